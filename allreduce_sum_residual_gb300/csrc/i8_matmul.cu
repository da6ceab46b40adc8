// ar_i8_matmul: checks and the choice of kernel.
#include "i8_matmul.cuh"

namespace arn {

struct I8Plan {
  int tokens;  // of a tile; 0: the matvec kernel
  int split;
};

static I8Plan i8_plan(int64_t m, int64_t width, int64_t K, bool gated, int sms, const int *pairs) {
  if (m <= 8) return {0, 1};
  const int64_t channels = gated ? 64 : 128;
  const int64_t tiles_n = (width + channels - 1) / channels, steps = (K + 127) / 128;
  if (m > 128) {
    const int64_t tiles = (tiles_n + 1) / 2 * ((m + 255) / 256);
    if (tiles * 4 >= pairs[0] * 3) return {256, 1};
  }
  const int tokens = m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 ? 64 : 128;
  const int64_t tiles = tiles_n * ((m + tokens - 1) / tokens);
  const int64_t slots = static_cast<int64_t>(sms) * (tokens <= 64 ? 2 : 1);
  int split = 1;
  while (split < 8 && tiles * split * 2 <= slots && steps >= 4 * split) split *= 2;
  return {tokens, split};
}

static int run_i8_matmul(const int8_t *x, const float *x_scales, const int8_t *w,
                         const float *w_scales, int64_t m, int64_t N, int64_t K, int act,
                         int out_type, void *out, void *stream) {
  const int size = type_size(out_type);
  if (m < 0 || N < 1 || K < 1 || size == 0 || (act != AR_ACT_NONE && act != AR_ACT_SILU_MUL) ||
      (act == AR_ACT_SILU_MUL && N % 2 != 0))
    return AR_ERR_ARG;
  if (K % 16 != 0) return AR_ERR_ALIGN;
  if (K > AR_I8_MAX_K || N > AR_I8_MAX_N || m > AR_I8_MAX_ROWS) return AR_ERR_UNSUPPORTED;
  if (m == 0) return AR_OK;
  if (!x || !x_scales || !w || !w_scales || !out) return AR_ERR_ARG;
  if (!aligned16(x) || !aligned16(w) || !aligned_to(x_scales, 4) || !aligned_to(w_scales, 4) ||
      !aligned_to(out, size))
    return AR_ERR_ALIGN;
  const int64_t width = act == AR_ACT_SILU_MUL ? N / 2 : N;
  const Range o = range_of(out, m * width * size);
  if (overlap(o, range_of(x, m * K)) || overlap(o, range_of(x_scales, m * 4)) ||
      overlap(o, range_of(w, N * K)) || overlap(o, range_of(w_scales, N * 4)))
    return AR_ERR_ALIAS;
  int st;
  DeviceState *d = current_device(&st);
  if (!d) return st;
  I8Args a = {};
  a.x = x;
  a.xs = x_scales;
  a.w = w;
  a.ws = w_scales;
  a.out = out;
  a.m = m;
  a.width = width;
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(K);
  a.gated = act == AR_ACT_SILU_MUL;
  a.out_type = out_type;
  a.status = d->status;
  const int *pairs = nullptr;
  st = ready_i8_tensor(d->sms, &pairs);
  if (st != AR_OK) return st;
  const cudaStream_t on = static_cast<cudaStream_t>(stream);
  const I8Plan p = i8_plan(m, width, K, a.gated, d->sms, pairs);
  if (p.tokens == 0)
    return launch_i8_matvec(a, d->sms, on) == cudaSuccess ? AR_OK : AR_ERR_CUDA;
  return launch_i8_tensor(a, p.tokens, p.split, pairs[0], on);
}

}  // namespace arn

using namespace arn;

extern "C" {

int ar_i8_matmul(const int8_t *x, const float *x_scales, const int8_t *w, const float *w_scales,
                 int64_t m, int64_t N, int64_t K, int act, int out_type, void *out, void *stream) {
  return run_i8_matmul(x, x_scales, w, w_scales, m, N, K, act, out_type, out, stream);
}

}  // extern "C"
