// The norms after and before a block, with its gate and the residual's and
// the block's scales (ar_block_rmsnorm and ar_block_rmsnorm_i8): the kernel.
//
//   s = sum_k p_k                       b = s / rms(s) (pw + off)   (with pw)
//   r = rscale res + bscale gate b      y = r / rms(r) (w + off)
//   out = y, or bytes q = round(127 y / max|y|) with the row's max|y| / 127
//
// Bound by memory: a row's n + 1 inputs are read once, r and y written once,
// and everything between stays in the registers of the threads that hold the
// row, a pack each.  Two sums over the row stand between its loads and its
// stores, where the epilogue without a norm after the block has one: sum r^2
// could be had together with sum s^2 from sums of s^2, res^2 and s res, but
// where the block and the residual nearly cancel that leaves nothing but
// their roundings, so it is summed from r itself.  The largest |y| is found
// in the same pass as sum r^2: 1 / rms(r) multiplies the whole row, so the
// bytes come from r (w + off) alone and the scale takes the factor.
//
// The split is the fused epilogue's: a CTA a row, or a cluster of them where
// there are few rows.
#pragma once

#include "dense.cuh"

namespace arn {

struct BlockNormArgs {
  const uint4 *p[AR_MAX_RANKS];  // [m, P] packs
  const uint4 *post;             // [P], or null
  const uint4 *gate;             // rows of P packs, or null
  const uint4 *res;              // [m, P] packs, twice as many in fp32
  const uint4 *w;                // [P]
  void *out;                     // [m, P] packs of 16 bytes, or of 8 (bytes)
  float *scales;                 // [m], or null: 16-bit output
  uint4 *rout;                   // as res
  int64_t m;
  int64_t gate_stride;           // packs
  int64_t gate_rows;             // rows of out that share a row of gate
  int n, P, per_cta, split;
  int64_t ahead;                 // rows to prefetch ahead (one CTA a row); 0: none
  float H, eps, block_scale, residual_scale, offset;
  uint64_t wait_limit_ns;
  int *status;
};

// What the CTAs of a cluster tell one another, twice a row.
struct BlockNormShared {
  float red[2][33];
  uint32_t redm[33];
  float totals[2][kMaxClusterCtas];
  float tops[kMaxClusterCtas];
  uint64_t bar[2];
  int abort;
};

// A sum over the row (and, with `top`, the largest of its bits), from the
// CTA's threads and then the CTAs of its cluster in rank order.
template <bool CL>
__device__ __forceinline__ float row_sum(float v, uint32_t *top, int round, uint32_t q, uint32_t S,
                                         BlockNormShared &sh, const BlockNormArgs &a) {
  if (top != nullptr) {  // ordered by block_sum's barrier
    const uint32_t warp_top = __reduce_max_sync(0xFFFFFFFFu, *top);
    if ((threadIdx.x & 31) == 0) sh.redm[threadIdx.x >> 5] = warp_top;
  }
  float total = block_sum(v, sh.red[round]);
  if (top != nullptr) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    *top = __reduce_max_sync(0xFFFFFFFFu, lane < warps ? sh.redm[lane] : 0u);
  }
  if constexpr (CL) {
    if (round == 0 || a.post == nullptr) cluster_wait_acquire();  // once: every CTA runs
    if (threadIdx.x == 0)
      mbar_arrive_expect_tx(&sh.bar[round], S * (top != nullptr ? 8u : 4u));
    if (threadIdx.x < S) {
      st_async_remote_f32(&sh.totals[round][q], threadIdx.x, total, &sh.bar[round]);
      if (top != nullptr)
        st_async_remote_f32(&sh.tops[q], threadIdx.x, __uint_as_float(*top), &sh.bar[round]);
    }
    mbar_wait_bounded(&sh.bar[round], 0, &sh.abort, a.wait_limit_ns, a.status);
    total = 0.f;
    for (uint32_t s = 0; s < S; ++s) total += sh.totals[round][s];
    if (top != nullptr) {
      uint32_t t = 0;
      for (uint32_t s = 0; s < S; ++s) t = max(t, __float_as_uint(sh.tops[s]));
      *top = t;
    }
  }
  return total;
}

// T: bf16 or fp16.  R32: the residual is fp32.  Threads of a CTA at most,
// CTAs of an SM at least (the register budget).  CL: a cluster a row.
template <typename T, bool R32, int THREADS, int CTAS, bool CL>
__global__ void __launch_bounds__(THREADS, CTAS)
    k_block_norm(const __grid_constant__ BlockNormArgs a) {
  __shared__ BlockNormShared sh;
  constexpr int U = 4;  // rows of partials in flight
  const uint32_t S = static_cast<uint32_t>(a.split);
  const uint32_t q = CL ? cluster_ctarank() : 0;
  const int64_t row = CL ? blockIdx.x / S : blockIdx.x;
  const int c0 = static_cast<int>(q) * a.per_cta;
  const int c1 = min(a.P, c0 + a.per_cta);
  const int64_t base = row * static_cast<int64_t>(a.P);
  // Checking build: the row, its pack range, and threads for all of it.
  const bool live = in_bounds(row < a.m && c0 >= 0 &&
                                  (c1 <= c0 || c1 - c0 <= static_cast<int>(blockDim.x)) &&
                                  a.n >= 1 && a.n <= AR_MAX_RANKS &&
                                  (!CL || S <= static_cast<uint32_t>(kMaxClusterCtas)) && q < S,
                              a.status);
  if constexpr (CL) {
    if (threadIdx.x == 0) {
      mbar_init(&sh.bar[0], 1);
      mbar_init(&sh.bar[1], 1);
      sh.abort = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    cluster_arrive_release();
  }
  pdl_wait_prior_grid();
  pdl_launch_dependents();

  const int c = c0 + static_cast<int>(threadIdx.x);
  const bool in = live && c < c1;
  const uint4 none = make_uint4(0, 0, 0, 0);
  const int64_t gate_at = a.gate != nullptr ? row / a.gate_rows * a.gate_stride + c : 0;
  // Clusters load everything at once (fewer trips in a row); one CTA a row
  // loads the factors late (fewer registers, more CTAs an SM).
  uint4 pw = none, gv = none, wv = none, r0 = none, r1 = none;
  if constexpr (CL) {
    if (in) {
      if (a.post != nullptr) pw = ld_ro(a.post + c);
      if (a.gate != nullptr) gv = ld_ro(a.gate + gate_at);
      wv = ld_ro(a.w + c);
      r0 = ld_ro(a.res + (base + c) * (R32 ? 2 : 1));
      if (R32) r1 = ld_ro(a.res + (base + c) * 2 + 1);
    }
  }
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int k0 = 0; k0 < a.n; k0 += U) {
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      x[u] = none;
      if (in && k0 + u < a.n) x[u] = ld_ro(a.p[k0 + u] + base + c);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[8];
      unpack16<T>(x[u], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += f[e];
    }
  }
  if constexpr (!CL) {
    if (in) {
      r0 = ld_ro(a.res + (base + c) * (R32 ? 2 : 1));
      if (R32) r1 = ld_ro(a.res + (base + c) * 2 + 1);
    }
    // The same rows one wave of CTAs ahead, on their way to L2.
    const int t = threadIdx.x;
    if (live && a.ahead > 0 && row + a.ahead < a.m && t <= a.n) {
      const uint32_t bytes = static_cast<uint32_t>(a.P) * 16u;
      const int64_t at = base + a.ahead * a.P;
      if (t < a.n)
        prefetch_l2(a.p[t] + at, bytes);
      else
        prefetch_l2(a.res + at * (R32 ? 2 : 1), R32 ? 2 * bytes : bytes);
    }
  }
  if (a.post != nullptr) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(acc[e], acc[e], ss);
    if constexpr (!CL) {
      if (in) pw = ld_ro(a.post + c);
    }
    const float total = row_sum<CL>(ss, nullptr, 0, q, S, sh, a);
    const float inv = rsqrtf(total / a.H + a.eps);
    float f[8];
    unpack16<T>(pw, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = (acc[e] * inv) * (f[e] + a.offset);
  }
  if (a.gate != nullptr) {
    if constexpr (!CL) {
      if (in) gv = ld_ro(a.gate + gate_at);
    }
    float f[8];
    unpack16<T>(gv, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] *= f[e];
  }
  {
    float f[8];
    if constexpr (R32) {
      const uint32_t w[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(w[e]);
    } else {
      unpack16<T>(r0, f);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = fmaf(acc[e], a.block_scale, f[e] * a.residual_scale);
  }
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) ss = fmaf(acc[e], acc[e], ss);
  if (in) {
    if constexpr (R32) {
      uint4 *to = a.rout + (base + c) * 2;
      st_stream(to, make_uint4(__float_as_uint(acc[0]), __float_as_uint(acc[1]),
                               __float_as_uint(acc[2]), __float_as_uint(acc[3])));
      st_stream(to + 1, make_uint4(__float_as_uint(acc[4]), __float_as_uint(acc[5]),
                                   __float_as_uint(acc[6]), __float_as_uint(acc[7])));
    } else {
      st_stream(a.rout + base + c, pack16<T>(acc));
    }
  }
  if constexpr (!CL) {
    if (in) wv = ld_ro(a.w + c);
  }
  if (a.scales == nullptr) {
    const float total = row_sum<CL>(in ? ss : 0.f, nullptr, 1, q, S, sh, a);
    const float inv = rsqrtf(total / a.H + a.eps);
    float f[8];
    unpack16<T>(wv, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = (acc[e] * inv) * (f[e] + a.offset);
    if (in) st_stream(static_cast<uint4 *>(a.out) + base + c, pack16<T>(f));
    return;
  }
  // In bytes.  A row whose norm holds anything that is not finite gets zeros
  // and a scale of NaN.
  {
    float f[8];
    unpack16<T>(wv, f);
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      acc[e] *= f[e] + a.offset;
      top = max(top, magnitude_bits(acc[e]));
    }
    if (!in) top = 0;
    const float total = row_sum<CL>(in ? ss : 0.f, &top, 1, q, S, sh, a);
    const float inv = rsqrtf(total / a.H + a.eps);
    const float most = __uint_as_float(top);
    const float scale = most * inv / 127.f;
    const bool fine = top < kInfinityBits && magnitude_bits(scale) < kInfinityBits;
    // 2^100 keeps the quotient finite for rows of tiny values.
    const float up = most < 0x1p-100f ? 0x1p100f : 1.f;
    const float by = fine && top != 0 ? 127.f / (most * up) : 0.f;
    float b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = fmaf(fine ? acc[e] * up : 0.f, by, kRoundingBias);
    if (in) {
      const uint2 v = make_uint2(bytes_of_biased(b[0], b[1], b[2], b[3]),
                                 bytes_of_biased(b[4], b[5], b[6], b[7]));
      __stcs(static_cast<uint2 *>(a.out) + base + c, v);
    }
    if (live && q == 0 && threadIdx.x == 0)
      a.scales[row] = fine ? scale : __uint_as_float(0x7FC00000u);
  }
}

using BlockNormKernel = void (*)(BlockNormArgs);

// The kernel for rows of `threads` threads a CTA; *ctas: CTAs of an SM that
// its register budget keeps.
BlockNormKernel block_norm_bf16(bool r32, bool cluster, int threads, int *ctas);
BlockNormKernel block_norm_f16(bool r32, bool cluster, int threads, int *ctas);

template <typename T>
inline BlockNormKernel block_norm_of(bool r32, bool cluster, int threads, int *ctas) {
  *ctas = threads <= 512 ? 1536 / threads : threads <= 768 ? 2 : 2;
  if (*ctas > 32) *ctas = 32;
  if (cluster) return r32 ? &k_block_norm<T, true, 1024, 1, true> : &k_block_norm<T, false, 1024, 1, true>;
  if (threads <= 512)
    return r32 ? &k_block_norm<T, true, 512, 3, false> : &k_block_norm<T, false, 512, 3, false>;
  if (threads <= 768)
    return r32 ? &k_block_norm<T, true, 768, 2, false> : &k_block_norm<T, false, 768, 2, false>;
  return r32 ? &k_block_norm<T, true, 1024, 2, false> : &k_block_norm<T, false, 1024, 2, false>;
}

}  // namespace arn
