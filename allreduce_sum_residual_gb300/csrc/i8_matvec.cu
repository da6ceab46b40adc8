// Products of a few rows with 8-bit weights: ar_i8_matmul where there are too
// few tokens to fill a tensor core's tile.
//
// Bound by the weights' bytes.  A warp takes a block of four weight rows, or
// two gate rows with their two up rows, and reads them as they lie, 16 bytes a
// lane; x comes through L1, where its few rows stay.  Each word of four
// weights costs one dp4a a token: with MT tokens MT / 4 operations a byte of
// weights, of which memory brings an SM some 24 a clock.  Sums are int32 and
// exact (K 2^14 < 2^31), so neither the order nor the split matters.
//
// The warps of a team share a row block, each a part of K, so that short
// matrices still give every SM its warps.
//
// Measured, one token: 7168 x 7168 in 9.1 us (5.7 TB/s; 3 us of it the launch and
// the first bytes), 32768 x 6144 gated in 30.3 us (6.6 TB/s), 8192 x 1024 in 2.7 us.
// With more than four tokens the dp4a are the bound (some 33 lanes a clock and SM):
// 8 x 7168 x 7168 takes 20.8 us, on the tensor cores 15.2 us (six calls a graph).
#include "i8_matmul.cuh"

namespace arn {

constexpr int kVecWarps = 8;
constexpr int kVecRows = 4;
// Bytes of a row, for each warp of its team, that are prefetched before the
// previous grid's end: one token through 7168 x 7168 takes 9.1 us, 11.2 us without
// and 11.5 us where the whole row is.
constexpr int kVecPrefetch = 1536;

__device__ __forceinline__ int4 ld_stream16(const int8_t *p) {
  int4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ int dot16(const int4 &a, const int4 &b, int c) {
  c = __dp4a(a.x, b.x, c);
  c = __dp4a(a.y, b.y, c);
  c = __dp4a(a.z, b.z, c);
  return __dp4a(a.w, b.w, c);
}

template <int MT, bool GATED>
__global__ void __launch_bounds__(kVecWarps * 32)
    k_i8_matvec(const __grid_constant__ I8Args a) {
  __shared__ int part[kVecWarps][kVecRows * MT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = warp % a.team;
  constexpr int kOuts = GATED ? kVecRows / 2 : kVecRows;
  const int64_t block = static_cast<int64_t>(blockIdx.x / a.token_blocks) * (kVecWarps / a.team) + warp / a.team;
  const int64_t j0 = block * kOuts;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x % a.token_blocks) * MT;
  // Rows and tokens behind the last take the last one's place; their sums
  // are not stored.
  const int8_t *wp[kVecRows], *xp[MT];
#pragma unroll
  for (int r = 0; r < kVecRows; ++r) {
    const int64_t j = min(j0 + (GATED ? r / 2 : r), a.width - 1) + (GATED && (r & 1) ? a.width : 0);
    wp[r] = a.w + j * a.K;
  }
  // The first bytes of the team's rows, on their way to L2 while the previous grid
  // ends.
  if (sub == 0 && lane == 0 && j0 < a.width) {
    const uint32_t bytes = static_cast<uint32_t>(min(a.K, kVecPrefetch * a.team));
#pragma unroll
    for (int r = 0; r < kVecRows; ++r) {
      if (in_bounds(wp[r] + a.K <= a.w + static_cast<int64_t>(a.N) * a.K, a.status))
        prefetch_l2(wp[r], bytes);
    }
  }
  pdl_wait_prior_grid();
  pdl_launch_dependents();
#pragma unroll
  for (int t = 0; t < MT; ++t) xp[t] = a.x + min(i0 + t, a.m - 1) * a.K;
  int acc[kVecRows][MT];
#pragma unroll
  for (int r = 0; r < kVecRows; ++r) {
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[r][t] = 0;
  }
  if (in_bounds(a.team >= 1 && kVecWarps % a.team == 0 && i0 < a.m, a.status)) {
    const int step = a.team * 512;
    int k = (sub * 32 + lane) * 16;
    for (; k + step < a.K; k += 2 * step) {
      int4 w0[kVecRows], w1[kVecRows];
#pragma unroll
      for (int r = 0; r < kVecRows; ++r) {
        w0[r] = ld_stream16(wp[r] + k);
        w1[r] = ld_stream16(wp[r] + k + step);
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int4 x0 = __ldg(reinterpret_cast<const int4 *>(xp[t] + k));
        const int4 x1 = __ldg(reinterpret_cast<const int4 *>(xp[t] + k + step));
#pragma unroll
        for (int r = 0; r < kVecRows; ++r)
          acc[r][t] = dot16(w1[r], x1, dot16(w0[r], x0, acc[r][t]));
      }
    }
    if (k < a.K) {
      int4 w0[kVecRows];
#pragma unroll
      for (int r = 0; r < kVecRows; ++r) w0[r] = ld_stream16(wp[r] + k);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int4 x0 = __ldg(reinterpret_cast<const int4 *>(xp[t] + k));
#pragma unroll
        for (int r = 0; r < kVecRows; ++r) acc[r][t] = dot16(w0[r], x0, acc[r][t]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kVecRows; ++r) {
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int v = __reduce_add_sync(0xFFFFFFFFu, acc[r][t]);
      if (lane == 0) part[warp][r * MT + t] = v;
    }
  }
  __syncthreads();
  if (sub != 0 || lane >= kOuts * MT) return;
  const int o = lane / MT, t = lane % MT;
  const int64_t i = i0 + t, j = j0 + o;
  if (i >= a.m || j >= a.width) return;
  const float xs = __ldg(a.xs + i);
  float v[2];
#pragma unroll
  for (int h = 0; h < (GATED ? 2 : 1); ++h) {
    const int r = GATED ? 2 * o + h : o;
    int s = 0;
    for (int u = 0; u < a.team; ++u) s += part[warp + u][r * MT + t];
    v[h] = static_cast<float>(s) * __ldg(a.ws + j + (h ? a.width : 0)) * xs;
  }
  if (in_bounds(i * a.width + j < a.m * a.width && warp + a.team <= kVecWarps, a.status))
    i8_store(a, i * a.width + j, GATED ? silu_mul(v[0], v[1]) : v[0]);
}

using MatvecKernel = void (*)(I8Args);

cudaError_t launch_i8_matvec(I8Args a, int sms, cudaStream_t stream) {
  const int mt = a.m <= 1 ? 1 : a.m <= 2 ? 2 : a.m <= 4 ? 4 : 8;
  const MatvecKernel kern =
      a.gated ? (mt == 1   ? &k_i8_matvec<1, true>
                 : mt == 2 ? &k_i8_matvec<2, true>
                 : mt == 4 ? &k_i8_matvec<4, true>
                           : &k_i8_matvec<8, true>)
              : (mt == 1   ? &k_i8_matvec<1, false>
                 : mt == 2 ? &k_i8_matvec<2, false>
                 : mt == 4 ? &k_i8_matvec<4, false>
                           : &k_i8_matvec<8, false>);
  const int outs = a.gated ? kVecRows / 2 : kVecRows;
  const int64_t blocks = (a.width + outs - 1) / outs;
  // A team grows while the row blocks leave an SM below sixteen warps and
  // each of its warps keeps two steps of 512.
  a.team = 1;
  while (a.team < kVecWarps && blocks * a.team < 16LL * sms && a.K >= 2 * a.team * 512) a.team *= 2;
  const int64_t per_cta = kVecWarps / a.team;
  a.token_blocks = static_cast<int>((a.m + mt - 1) / mt);
  const int64_t grid = (blocks + per_cta - 1) / per_cta;
  if (grid > INT32_MAX / a.token_blocks) return cudaErrorInvalidConfiguration;
  return launch_pdl(kern, a, grid * a.token_blocks, kVecWarps * 32, 0, 1, stream);
}

}  // namespace arn
