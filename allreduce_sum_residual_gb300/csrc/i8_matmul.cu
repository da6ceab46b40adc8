// ar_i8_matmul: checks and the choice of kernel.
#include "i8_matmul.cuh"

namespace arn {

struct I8Plan {
  int tokens;  // of a tile; 0: the matvec kernel
  int split;   // parts of K
};

// Microseconds, fitted to 1000 times of 230 shapes (1 to 2048 tokens, matrices of
// 512 x 512 to 32768 x 6144); the choice by them is within 2 % of the best on
// average, 14 % at most.
struct I8Cost {
  int tokens;
  double fixed;   // of a launch
  double join;    // each doubling of the split
  double alone;   // a stage of 128 k of one CTA on an SM
  double shared;  // and of each of several
};
constexpr I8Cost kI8Costs[] = {{16, 4.5, 0.5, 0.32, 0.32},
                               {32, 4.6, 0.7, 0.37, 0.31},
                               {64, 5.3, 0.9, 0.56, 0.40},
                               {128, 4.5, 3.1, 0.60, 0.60}};
constexpr double kI8Round = 6.8;                       // another tile behind one, one CTA a tile
constexpr I8Cost kI8Pair = {256, 2.0, 1.6, 0.54, 0.54};
constexpr double kI8PairTile = 6.3, kI8PairGated = 7.9;  // a pair's tile beside its stages

static I8Plan i8_plan(int64_t m, int64_t width, int64_t N, int64_t K, bool gated, int sms,
                      const int *pairs) {
  const int64_t channels = gated ? 64 : 128, steps = (K + 127) / 128;
  I8Plan best = {0, 1};
  double least = 1e30;
  if (m <= 16)  // bytes a microsecond of weights, once for eight tokens
    least = 3.2 + static_cast<double>((m + 7) / 8 * N * K) / (m <= 2 ? 6.0e6 : m <= 4 ? 4.3e6 : 2.8e6);
  for (const I8Cost &c : kI8Costs) {
    if (c.tokens < m && c.tokens < 128 && m > 4 * c.tokens) continue;
    if (c.tokens >= 2 * m && c.tokens > 16) break;
    const int64_t tiles = (width + channels - 1) / channels * ((m + c.tokens - 1) / c.tokens);
    const int at_a_time = c.tokens <= 64 ? 2 : 1;
    for (int split = 1; split <= 8 && split <= steps; split *= 2) {
      const int64_t on_sm = (tiles * split + sms - 1) / sms;
      const double stages = static_cast<double>((steps + split - 1) / split);
      const double t = c.fixed + (split == 1 ? 0 : split == 2 ? 1 : split == 4 ? 2 : 3) * c.join +
                       stages * (on_sm == 1 ? c.alone : on_sm * c.shared) +
                       static_cast<double>((on_sm - 1) / at_a_time) * kI8Round;
      if (t < least) {
        least = t;
        best = {c.tokens, split};
      }
    }
  }
  if (m > 64) {
    const int64_t tiles = (width + 2 * channels - 1) / (2 * channels) * ((m + 255) / 256);
    for (int i = 0; i < 3 && (1 << i) <= steps; ++i) {
      if (i > 0 && tiles > pairs[i]) break;  // a split's clusters take one tile each
      const int64_t rounds = (tiles + pairs[i] - 1) / pairs[i];
      const double stages = static_cast<double>((steps + (1 << i) - 1) >> i);
      const double t = kI8Pair.fixed + i * kI8Pair.join +
                       rounds * (stages * kI8Pair.alone + (gated ? kI8PairGated : kI8PairTile));
      if (t < least) {
        least = t;
        best = {256, 1 << i};
      }
    }
  }
  return best;
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
  const I8Plan p = i8_plan(m, width, N, K, a.gated, d->sms, pairs);
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
