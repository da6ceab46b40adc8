// Activations in 8 bits with a scale for each row (ar_i8_quantize).
//
//   scale_i = max_k |x_ik| / 127        q_ik = round(x_ik 127 / max_k |x_ik|)
//
// Bound by memory: two bytes read and one written a value (4096 rows of 16384:
// 29.8 us, a plain copy's rate).  A CTA takes a row and keeps it in registers, a
// thread VPT packs, from the loads through the row's maximum to the stores.
//
// Halves to even, decided as on the exact quotient, which fp32 can do for
// 16-bit x: with x = X 2^e and max = A 2^f, X and A of at most 11 bits, the
// quotient t differs from n + 1/2 by |254 X 2^e - (2n + 1) A 2^f| over
// 2 A 2^f, which is 0 or at least t / (254 X) > 2^-19 t.
//   - Where 127 does not divide A it is 0 only for 2n + 1 = 127, t = 63.5,
//     whose even neighbour is 64.  So one multiply-add by a reciprocal rounded
//     up (by less than 2^-22) decides everything: t = 63.5 goes up, and nothing
//     else is near enough to a border to be carried over it.
//   - Where 127 divides A any half may be met.  The product with the rounded
//     reciprocal is within 2^-23 t of the quotient; where twice it is within
//     2^-21 of itself of a whole number, it is that number (no other quotient
//     is so near), and everywhere else it is on its own side of the border.
// The second way for every row takes 12 operations a value instead of 3, more
// than memory leaves time for (8192 rows of 8192: 38.3 us).
#include "dense.cuh"

namespace arn {

struct QuantizeArgs {
  const uint4 *x;     // rows of P packs, `stride` packs apart
  uint2 *q;           // [m, P] packs of eight bytes
  float *scales;      // [m]
  int64_t m, stride;
  int64_t ahead;      // rows to prefetch ahead; 0: none
  int P;
  int *status;
};

// Twice the quotient as a whole number where it is one.
__device__ __forceinline__ float biased_quotient(float x, float by2) {
  const float t = x * by2;
  const float h = (t + kRoundingBias) - kRoundingBias;
  return fmaf(fabsf(t - h) <= fabsf(t) * 0x1p-21f ? h : t, 0.5f, kRoundingBias);
}

struct RowScale {
  bool plain;            // one multiply-add by `by`
  bool fine;
  float by, up, by2, scale;
};

// From the bits of the row's largest magnitude in fp32.  A row that holds
// anything that is not finite gets zeros and a scale of NaN.  2^100 keeps the
// reciprocal finite for rows of tiny values.
__device__ __forceinline__ RowScale row_scale(uint32_t top) {
  RowScale s;
  const float most = __uint_as_float(top);
  s.fine = top < kInfinityBits;
  s.plain = s.fine && most >= 0x1p-100f && ((top >> 13 & 0x3FFu) | 0x400u) % 127u != 0;
  s.by = __uint_as_float(__float_as_uint(127.f / most) + 1u);
  s.up = most < 0x1p-100f ? 0x1p100f : 1.f;
  s.by2 = s.fine && top != 0 ? 254.f / (most * s.up) : 0.f;
  s.scale = s.fine ? most / 127.f : __uint_as_float(0x7FC00000u);
  return s;
}

// The larger magnitudes of two pairs of 16-bit values, as bits: their order is
// that of the magnitudes, infinity above every number and NaN above infinity.
__device__ __forceinline__ uint32_t pair_top(uint32_t top, uint32_t x) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(top), "r"(x & 0x7FFF7FFFu));
  return r;
}
__device__ __forceinline__ uint32_t pack_top(const uint4 &x, uint32_t top) {
  return pair_top(pair_top(pair_top(pair_top(top, x.x), x.y), x.z), x.w);
}
template <typename T>
__device__ __forceinline__ uint32_t top_bits(uint32_t pair);
template <>
__device__ __forceinline__ uint32_t top_bits<__nv_bfloat16>(uint32_t pair) {
  return max(pair << 16, pair & 0xFFFF0000u);
}
template <>
__device__ __forceinline__ uint32_t top_bits<__half>(uint32_t pair) {
  const uint32_t h = max(pair & 0xFFFFu, pair >> 16);
  return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(h))));
}

template <typename T>
__device__ __forceinline__ void store_bytes(const QuantizeArgs &a, int64_t at, const uint4 &x,
                                            const RowScale &s) {
  float f[8];
  unpack16<T>(x, f);
  if (s.plain) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = fmaf(f[e], s.by, kRoundingBias);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = biased_quotient(s.fine ? f[e] * s.up : 0.f, s.by2);
  }
  __stcs(a.q + at, make_uint2(bytes_of_biased(f[0], f[1], f[2], f[3]),
                              bytes_of_biased(f[4], f[5], f[6], f[7])));
}

// VPT packs a thread in registers; 0: rows of any length, read twice.
template <typename T, int VPT, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS)
    k_i8_quantize(const __grid_constant__ QuantizeArgs a) {
  __shared__ uint32_t red[33];
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const int64_t row = blockIdx.x;
  const int T0 = threadIdx.x, step = blockDim.x;
  const bool live =
      in_bounds(row < a.m && (VPT == 0 || a.P <= static_cast<int>(blockDim.x) * VPT), a.status);
  const uint4 *from = a.x + row * a.stride;
  const int end = live ? a.P : 0;
  // The row one wave of CTAs ahead, on its way to L2.
  if (live && T0 == 0 && a.ahead > 0 && row + a.ahead < a.m)
    prefetch_l2(from + a.ahead * a.stride, static_cast<uint32_t>(a.P) * 16u);
  RowScale s;
  uint32_t top = 0;
  if constexpr (VPT == 0) {
    for (int c = T0; c < end; c += step) top = pack_top(ld_ro(from + c), top);
    s = row_scale(block_max(top_bits<T>(top), red));
    for (int c = T0; c < end; c += step) store_bytes<T>(a, row * a.P + c, ld_ro(from + c), s);
  } else {
    uint4 x[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      x[v] = make_uint4(0, 0, 0, 0);
      if (T0 + v * step < end) x[v] = ld_ro(from + T0 + v * step);
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) top = pack_top(x[v], top);
    s = row_scale(block_max(top_bits<T>(top), red));
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (T0 + v * step < end) store_bytes<T>(a, row * a.P + T0 + v * step, x[v], s);
    }
  }
  if (live && T0 == 0) a.scales[row] = s.scale;
}

using QuantizeKernel = void (*)(QuantizeArgs);

template <typename T>
static QuantizeKernel quantize_kernel(int vpt) {
  switch (vpt) {
    case 2: return &k_i8_quantize<T, 2, 512, 2>;
    case 4: return &k_i8_quantize<T, 4, 512, 2>;
    case 8: return &k_i8_quantize<T, 8, 512, 2>;
    default: return &k_i8_quantize<T, 0, 1024, 2>;
  }
}

static int run_quantize(const void *x, int type, int64_t row_stride, int64_t m, int64_t K, int8_t *q,
                        float *scales, void *stream) {
  if (m < 0 || K < 1 || !is_16bit(type) || row_stride < K) return AR_ERR_ARG;
  if (K % kPackElems != 0 || row_stride % kPackElems != 0) return AR_ERR_ALIGN;
  if (K > AR_MAX_HIDDEN || m > INT32_MAX || m > (int64_t{1} << 40) / row_stride)
    return AR_ERR_UNSUPPORTED;
  if (m == 0) return AR_OK;
  if (!x || !q || !scales) return AR_ERR_ARG;
  if (!aligned16(x) || !aligned16(q) || !aligned_to(scales, 4)) return AR_ERR_ALIGN;
  const Range in = range_of(x, ((m - 1) * row_stride + K) * 2);
  const Range o = range_of(q, m * K), s = range_of(scales, m * 4);
  if (overlap(o, in) || overlap(s, in) || overlap(o, s)) return AR_ERR_ALIAS;
  int st;
  DeviceState *d = current_device(&st);
  if (!d) return st;
  QuantizeArgs a = {};
  a.x = static_cast<const uint4 *>(x);
  a.q = reinterpret_cast<uint2 *>(q);
  a.scales = scales;
  a.m = m;
  a.stride = row_stride / kPackElems;
  a.P = static_cast<int>(K / kPackElems);
  a.status = d->status;
  // Four packs a thread where a row's CTA has 256 threads at most, else eight
  // (8192 rows of 4096: 16.1 us against 16.4 us; 4096 rows of 16384: 30.1 us
  // against 29.8 us); two where there are too few rows to fill the SMs (77 rows of
  // 5120: 2.4 us, with four 2.7 us).
  const bool few = m < 2 * d->sms;
  const int vpt = few && a.P <= 1024 ? 2 : a.P <= (few ? 2048 : 1024) ? 4 : a.P <= 4096 ? 8 : 0;
  const int threads = vpt == 0 ? 1024 : ((a.P + vpt - 1) / vpt + 31) / 32 * 32;
  const int ctas = 1024 / threads;  // 64 registers a thread
  if (!few) a.ahead = static_cast<int64_t>(d->sms) * (ctas > 32 ? 32 : ctas);
  const QuantizeKernel kern =
      type == AR_TYPE_BF16 ? quantize_kernel<__nv_bfloat16>(vpt) : quantize_kernel<__half>(vpt);
  return launch_pdl(kern, a, m, threads, 0, 1, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? AR_OK
             : AR_ERR_CUDA;
}

}  // namespace arn

using namespace arn;

extern "C" {

int ar_i8_quantize(const void *x, int type, int64_t row_stride, int64_t m, int64_t K, int8_t *q,
                   float *scales, void *stream) {
  return run_quantize(x, type, row_stride, m, K, q, scales, stream);
}

}  // extern "C"
