// Pieces shared by the calls of a dense layer in 8 bits (block_norm,
// i8_quantize, i8_matmul): 16-bit packs of either type and 8-bit rounding.
#pragma once

#include <cuda_fp16.h>

#include <cmath>

#include "experts.cuh"

namespace arn {

// A pack of eight 16-bit values of T (bf16 or fp16) as fp32, and back with
// one rounding to nearest even each.
template <typename T>
__device__ __forceinline__ void unpack16(const uint4 &v, float (&f)[8]);
template <>
__device__ __forceinline__ void unpack16<__nv_bfloat16>(const uint4 &v, float (&f)[8]) {
  unpack8(v, f);
}
template <>
__device__ __forceinline__ void unpack16<__half>(const uint4 &v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack16(const float (&f)[8]);
template <>
__device__ __forceinline__ uint4 pack16<__nv_bfloat16>(const float (&f)[8]) {
  return pack8(f);
}
template <>
__device__ __forceinline__ uint4 pack16<__half>(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 1.5 * 2^23: added to |t| < 2^22 it rounds t to a whole number, halves to
// even, whose low bits are the sum's low bits (two's complement).
constexpr float kRoundingBias = 12582912.f;

// Four values, already biased, as four signed bytes.
__device__ __forceinline__ uint32_t bytes_of_biased(float a, float b, float c, float d) {
  const uint32_t lo = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

// The bits of |v|, whose order as unsigned numbers is that of the
// magnitudes, infinity above every number and NaN above infinity.
__device__ __forceinline__ uint32_t magnitude_bits(float v) {
  return __float_as_uint(v) & 0x7FFFFFFFu;
}
constexpr uint32_t kInfinityBits = 0x7F800000u;

// The largest `v` of the CTA, returned to every thread; `scratch` holds 33
// words and is used once per kernel.
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t *scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nwarps = (blockDim.x + 31) >> 5;
  v = __reduce_max_sync(0xFFFFFFFFu, v);
  if (lane == 0) scratch[warp] = v;
  __syncthreads();
  return __reduce_max_sync(0xFFFFFFFFu, lane < nwarps ? scratch[lane] : 0u);
}

inline bool is_16bit(int type) { return type == AR_TYPE_BF16 || type == AR_TYPE_F16; }

}  // namespace arn
