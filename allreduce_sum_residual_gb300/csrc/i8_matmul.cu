// ar_i8_matmul: checks and the choice of kernel.
#include "i8_matmul.cuh"

namespace arn {

// Microseconds, fitted to the times of every shape of 341 products (1 to 2048
// tokens, matrices of 512 x 512 to 32768 x 6144), which profiles/ holds.  The choice
// by them takes 0.4 % longer than the best on average, 13 % at most (0.7 us).
struct I8Cost {
  int tokens;
  double fixed;   // of a launch
  double join;    // each doubling of the split
  double alone;   // a stage of 128 k of one CTA on an SM, or of a pair
  double shared;  // and of each of several CTAs
  double tile, gated;  // a pair's tile beside its stages
  int splits;     // 1 to 2^(splits - 1) parts of K
};
constexpr I8Cost kI8Ctas[] = {{16, 4.07, 0.51, 0.37, 0.33, 0, 0, 4}, {32, 4.31, 0.68, 0.40, 0.34, 0, 0, 4}};
constexpr double kI8Round = 5.28;  // another tile behind an SM's first two
constexpr I8Cost kI8Pairs[] = {{64, 4.17, 1.34, 0.37, 0, 0.67, 1.19, 2},
                               {128, 4.41, 0.84, 0.36, 0, 1.67, 2.40, 3},
                               {256, 4.56, 1.11, 0.56, 0, 3.72, 4.18, 3}};

// The launch shape for m tokens, and its microseconds.
static I8Plan i8_plan(int64_t m, int64_t width, int64_t N, int64_t K, bool gated, int sms,
                      const int *pairs, double *time) {
  const int64_t channels = gated ? 64 : 128, steps = (K + 127) / 128;
  I8Plan best = {0, 1, false};
  double least = 1e30;
  if (m <= 16) {  // dot products: the weights' bytes, once for eight tokens
    const double bytes = static_cast<double>((m + 7) / 8 * N * K);
    // Above eight tokens only the smallest matrices go there, and only they are fitted.
    least = m <= 2   ? 2.9 + bytes / 5.8e6
            : m <= 4 ? 3.0 + bytes / 3.7e6
            : m <= 8 ? 4.7 + bytes / 3.1e6
                     : 3.5 + bytes / 1.2e6;
  }
  // Two tokens at most never go faster on the tensor cores (two tokens, 32768 x 6144
  // gated: 32.4 us, with three there 33.9; 7168 x 7168: 9.0 and 12.7; one token, 57344
  // x 8192 gated: 64 us, there 82).
  if (m <= 2) {
    *time = least;
    return best;
  }
  for (const I8Cost &c : kI8Ctas) {
    if (m > 4 * c.tokens || (c.tokens > 16 && c.tokens >= 2 * m)) continue;
    const int64_t tiles = (width + channels - 1) / channels * ((m + c.tokens - 1) / c.tokens);
    for (int i = 0; i < c.splits && (1 << i) <= steps; ++i) {
      const int64_t on_sm = ((tiles << i) + sms - 1) / sms;
      const double stages = static_cast<double>((steps + (1 << i) - 1) >> i);
      const double t = c.fixed + i * c.join + stages * (on_sm == 1 ? c.alone : on_sm * c.shared) +
                       static_cast<double>((on_sm - 1) / 2) * kI8Round;
      if (t < least) {
        least = t;
        best = {c.tokens, 1 << i, false};
      }
    }
  }
  for (const I8Cost &c : kI8Pairs) {
    if (m <= c.tokens / 4) break;
    const int64_t tiles = (width + 2 * channels - 1) / (2 * channels) * ((m + c.tokens - 1) / c.tokens);
    for (int i = 0; i < c.splits && (1 << i) <= steps; ++i) {
      if (i > 0 && tiles > pairs[i]) break;  // a split's clusters take one tile each
      const int64_t rounds = i > 0 ? 1 : (tiles + pairs[0] - 1) / pairs[0];
      const double stages = static_cast<double>((steps + (1 << i) - 1) >> i);
      const double t = c.fixed + i * c.join +
                       static_cast<double>(rounds) * (stages * c.alone + (gated ? c.gated : c.tile));
      if (t < least) {
        least = t;
        best = {c.tokens, 1 << i, true};
      }
    }
  }
  *time = least;
  return best;
}

// Tokens to take first, by themselves: where the last round of 256-token tiles is
// far from full, the rest ends sooner as a launch of its own with smaller tiles
// (4096 x 16384 x 6144, 384 tiles for 76 pairs: 417 us, all at once 443 us).  0: all
// at once.
static int64_t i8_head(int64_t m, int64_t width, int64_t N, int64_t K, bool gated, int sms,
                       const int *pairs, const I8Plan &all, double time) {
  if (!all.pair || all.tokens != 256 || all.split != 1) return 0;
  int64_t head = 0;
  for (int64_t h = (m - 1) / 256 * 256, i = 0; h > 0 && i < 4; h -= 256, ++i) {
    double first, rest;
    const I8Plan p = i8_plan(h, width, N, K, gated, sms, pairs, &first);
    if (!p.pair || p.tokens != 256 || p.split != 1) break;
    i8_plan(m - h, width, N, K, gated, sms, pairs, &rest);
    // A launch less behind another, and 3 % for what the estimates are off by.
    if ((first + rest - 2.0) * 1.03 < time) {
      time = (first + rest - 2.0) * 1.03;
      head = h;
    }
  }
  return head;
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
  double time;
  I8Plan p = i8_plan(m, width, N, K, a.gated, d->sms, pairs, &time);
  if (p.tokens == 0) return launch_i8_matvec(a, d->sms, on) == cudaSuccess ? AR_OK : AR_ERR_CUDA;
  const int64_t head = i8_head(m, width, N, K, a.gated, d->sms, pairs, p, time);
  if (head > 0) {
    a.m = head;
    st = launch_i8_tensor(a, p, pairs[0], on);
    if (st != AR_OK) return st;
    a.m = m - head;
    a.x += head * K;
    a.xs += head;
    a.out = static_cast<char *>(a.out) + head * width * size;
    p = i8_plan(a.m, width, N, K, a.gated, d->sms, pairs, &time);
    if (p.tokens == 0) return launch_i8_matvec(a, d->sms, on) == cudaSuccess ? AR_OK : AR_ERR_CUDA;
  }
  return launch_i8_tensor(a, p, pairs[0], on);
}

}  // namespace arn

using namespace arn;

extern "C" {

int ar_i8_matmul(const int8_t *x, const float *x_scales, const int8_t *w, const float *w_scales,
                 int64_t m, int64_t N, int64_t K, int act, int out_type, void *out, void *stream) {
  return run_i8_matmul(x, x_scales, w, w_scales, m, N, K, act, out_type, out, stream);
}

}  // extern "C"
