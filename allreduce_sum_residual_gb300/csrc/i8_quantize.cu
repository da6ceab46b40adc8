// Activations in 8 bits with a scale for each row (ar_i8_quantize).
//
//   scale_i = max_k |x_ik| / 127        q_ik = round(x_ik 127 / max_k |x_ik|)
//
// Bound by memory: two bytes read and one written a value.  A CTA takes a
// row and keeps it in registers, a thread VPT packs, from the loads through
// the row's maximum to the stores.
//
// Halves to even, decided as on the exact quotient, which fp32 can do for
// 16-bit x: with x = X 2^e and max = A 2^f, X and A of at most 11 bits, the
// quotient t differs from n + 1/2 by |254 X 2^e - (2n + 1) A 2^f| over
// 2 A 2^f, which is 0 or at least t / (254 X) > 2^-19 t.  The product with
// the rounded reciprocal is within 2^-23 t of the quotient.  So where twice
// it is within 2^-21 of itself of a whole number, it is that number (no other
// quotient is so near), and everywhere else it is on its own side of the
// border.
#include "dense.cuh"

namespace arn {

struct QuantizeArgs {
  const uint4 *x;     // rows of P packs, `stride` packs apart
  uint2 *q;           // [m, P] packs of eight bytes
  float *scales;      // [m]
  int64_t m, stride;
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
  bool fine;
  float up, by2, scale;
};

// A row that holds anything that is not finite gets zeros and a scale of NaN.
// 2^100 keeps the reciprocal finite for rows of tiny values.
__device__ __forceinline__ RowScale row_scale(uint32_t top) {
  RowScale s;
  const float most = __uint_as_float(top);
  s.fine = top < kInfinityBits;
  s.up = most < 0x1p-100f ? 0x1p100f : 1.f;
  s.by2 = s.fine && top != 0 ? 254.f / (most * s.up) : 0.f;
  s.scale = s.fine ? most / 127.f : __uint_as_float(0x7FC00000u);
  return s;
}

template <typename T>
__device__ __forceinline__ uint32_t pack_top(const uint4 &x, uint32_t top) {
  float f[8];
  unpack16<T>(x, f);
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, magnitude_bits(f[e]));
  return top;
}

template <typename T>
__device__ __forceinline__ void store_bytes(const QuantizeArgs &a, int64_t at, const uint4 &x,
                                            const RowScale &s) {
  float f[8];
  unpack16<T>(x, f);
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = biased_quotient(s.fine ? f[e] * s.up : 0.f, s.by2);
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
  RowScale s;
  uint32_t top = 0;
  if constexpr (VPT == 0) {
    for (int c = T0; c < end; c += step) top = pack_top<T>(ld_ro(from + c), top);
    s = row_scale(block_max(top, red));
    for (int c = T0; c < end; c += step) store_bytes<T>(a, row * a.P + c, ld_ro(from + c), s);
  } else {
    uint4 x[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      x[v] = make_uint4(0, 0, 0, 0);
      if (T0 + v * step < end) x[v] = ld_ro(from + T0 + v * step);
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) top = pack_top<T>(x[v], top);
    s = row_scale(block_max(top, red));
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
    case 1: return &k_i8_quantize<T, 1, 1024, 2>;
    case 2: return &k_i8_quantize<T, 2, 512, 3>;
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
  int vpt = 1;
  if (a.P > 1024) {
    while (vpt <= 8 && (a.P + vpt - 1) / vpt > 512) vpt *= 2;
    if (vpt > 8) vpt = 0;
  }
  const int threads = vpt == 0 ? 1024 : ((a.P + vpt - 1) / vpt + 31) / 32 * 32;
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
