// The norms after and before a block, with its gate and the residual's and
// the block's scales (ar_block_rmsnorm and ar_block_rmsnorm_i8): the kernel.
//
//   s = sum_k p_k                       b = s / rms(s) (pw + off)   (with pw)
//   r = rscale res + bscale gate b      y = r / rms(r) (w + off)
//   out = y, or bytes q = round(127 y / max|y|) with the row's max|y| / 127
//
// Bound by memory: a row's n + 1 inputs are read once, r and y written once,
// and everything between stays in the registers of the threads that hold the
// row.  Two sums over the row stand between its loads and its stores, where the
// epilogue without a norm after the block has one: sum r^2 could be had together
// with sum s^2 from sums of s^2, res^2 and s res, but where the block and the
// residual nearly cancel that leaves nothing but their roundings, so it is summed
// from r itself.  The largest |y| is found in the same pass as sum r^2: 1 / rms(r)
// multiplies the whole row, so the bytes come from r (w + off) alone and the scale
// takes the factor.
//
// The split: a CTA a row with two or four packs a thread, or a cluster of them
// where there are few rows, or long ones.  The rows one wave of CTAs ahead are
// prefetched into L2 (8192 rows of 6144, one partial: 61.4 us, 6.56 TB/s; 78 us
// without the prefetch, 96 us with a pack a thread).  16 rows of 7168 and eight
// partials take 3.0 us from a graph: the launch, one trip to memory and two over
// the cluster.
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

// What the warps of a row tell one another, twice a row.
template <bool CL>
struct BlockNormShared {
  float red[2][33];
  uint32_t redm[33];
};
template <>
struct BlockNormShared<true> {
  float sums[2][kMaxClusterCtas * 32];
  float tops[kMaxClusterCtas * 32];
  uint64_t bar[2];
  int abort;
};

// A sum over the row (and, with `top`, the largest of its bits).
__device__ __forceinline__ float row_sum(float v, uint32_t *top, int round, uint32_t, uint32_t,
                                         BlockNormShared<false> &sh, const BlockNormArgs &) {
  if (top != nullptr) {  // ordered by block_sum's barrier
    const uint32_t warp_top = __reduce_max_sync(0xFFFFFFFFu, *top);
    if ((threadIdx.x & 31) == 0) sh.redm[threadIdx.x >> 5] = warp_top;
  }
  const float total = block_sum(v, sh.red[round]);
  if (top != nullptr) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    *top = __reduce_max_sync(0xFFFFFFFFu, lane < warps ? sh.redm[lane] : 0u);
  }
  return total;
}

// Over a cluster: every warp sends its sum to every CTA, and every warp adds
// all of them, in one order everywhere.  No barrier of the CTA stands between:
// with one, and a CTA's total sent, 16 rows of 7168 took 5.1 us.
__device__ __forceinline__ float row_sum(float v, uint32_t *top, int round, uint32_t q, uint32_t S,
                                         BlockNormShared<true> &sh, const BlockNormArgs &a) {
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (threadIdx.x == 0)
    mbar_arrive_expect_tx(&sh.bar[round], S * warps * (top != nullptr ? 8u : 4u));
  v = warp_sum(v);
  const uint32_t warp_top = top != nullptr ? __reduce_max_sync(0xFFFFFFFFu, *top) : 0u;
  if (round == 0 || a.post == nullptr) cluster_wait_acquire();  // once: every CTA runs
  if (lane < S) {
    st_async_remote_f32(&sh.sums[round][q * warps + warp], lane, v, &sh.bar[round]);
    if (top != nullptr)
      st_async_remote_f32(&sh.tops[q * warps + warp], lane, __uint_as_float(warp_top), &sh.bar[round]);
  }
  mbar_wait_bounded(&sh.bar[round], 0, &sh.abort, a.wait_limit_ns, a.status);
  float total = 0.f;
  uint32_t most = 0;
  for (uint32_t i = lane; i < S * warps; i += 32) {
    total += sh.sums[round][i];
    if (top != nullptr) most = max(most, __float_as_uint(sh.tops[i]));
  }
  if (top != nullptr) *top = __reduce_max_sync(0xFFFFFFFFu, most);
  return warp_sum(total);
}

// The eight values of a residual's pack.
template <typename T, bool R32>
__device__ __forceinline__ void unpack_residual(const uint4 (&r)[R32 ? 2 : 1], float (&f)[8]) {
  if constexpr (R32) {
    const uint32_t w[8] = {r[0].x, r[0].y, r[0].z, r[0].w, r[1].x, r[1].y, r[1].z, r[1].w};
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(w[e]);
  } else {
    unpack16<T>(r[0], f);
  }
}

// T: bf16 or fp16.  R32: the residual is fp32.  V: packs a thread.  Threads of
// a CTA at most, CTAs of an SM at least (the register budget).  CL: a cluster a
// row.
template <typename T, bool R32, int V, int THREADS, int CTAS, bool CL>
__global__ void __launch_bounds__(THREADS, CTAS)
    k_block_norm(const __grid_constant__ BlockNormArgs a) {
  __shared__ BlockNormShared<CL> sh;
  constexpr int kParts = R32 ? 2 : 1;           // 16-byte pieces of a residual's pack
  constexpr int U = V == 1 ? 8 : V == 2 ? 2 : 1;  // partials in flight
  // With one pack a thread a cluster loads everything at once (fewer trips in a
  // row); else the factors come late (fewer registers, more CTAs an SM), behind
  // the sums with four packs, and so does a residual in fp32 (1023 rows of 5128,
  // three partials: 17.3 us, 18.6 us with the partials).
  constexpr bool kEarly = CL && V == 1, kLate = V > 2, kLateResidual = !kEarly && R32;
  const uint32_t S = static_cast<uint32_t>(a.split);
  const uint32_t q = CL ? cluster_ctarank() : 0;
  const int64_t row = CL ? blockIdx.x / S : blockIdx.x;
  const int c0 = static_cast<int>(q) * a.per_cta;
  const int c1 = min(a.P, c0 + a.per_cta);
  const int64_t base = row * static_cast<int64_t>(a.P);
  const int T0 = threadIdx.x, step = blockDim.x;
  // Checking build: the row, its pack range, and threads for all of it.
  const bool live = in_bounds(row < a.m && c0 >= 0 && (c1 <= c0 || c1 - c0 <= step * V) && a.n >= 1 &&
                                  a.n <= AR_MAX_RANKS &&
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
  if (kEarly && live && c1 > c0 && threadIdx.x <= a.n) {
    // This CTA's part of the row, on its way to L2 while the previous grid ends.
    const uint32_t bytes = static_cast<uint32_t>(c1 - c0) * 16u;
    if (threadIdx.x < a.n)
      prefetch_l2(a.p[threadIdx.x] + base + c0, bytes);
    else
      prefetch_l2(a.res + (base + c0) * kParts, kParts * bytes);
  }
  pdl_wait_prior_grid();
  pdl_launch_dependents();

  const int end = live ? c1 : 0;
  const uint4 none = make_uint4(0, 0, 0, 0);
  const uint4 *gate = a.gate != nullptr ? a.gate + row / a.gate_rows * a.gate_stride : nullptr;
  uint4 pw[V], gv[V], wv[V], res[V][kParts];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    pw[v] = gv[v] = wv[v] = none;
#pragma unroll
    for (int i = 0; i < kParts; ++i) res[v][i] = none;
  }
  auto load = [&](uint4 (&to)[V], const uint4 *from) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = c0 + T0 + v * step;
      if (c < end) to[v] = ld_ro(from + c);
    }
  };
  auto load_residual = [&]() {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = c0 + T0 + v * step;
      if (c < end) {
#pragma unroll
        for (int i = 0; i < kParts; ++i) res[v][i] = ld_ro(a.res + (base + c) * kParts + i);
      }
    }
  };
  if constexpr (kEarly) {
    if (a.post != nullptr) load(pw, a.post);
    if (gate != nullptr) load(gv, gate);
    load(wv, a.w);
    load_residual();
  }
  float acc[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[v][e] = 0.f;
  }
  for (int k0 = 0; k0 < a.n; k0 += U) {
    uint4 x[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = c0 + T0 + v * step;
        x[u][v] = none;
        if (c < end && k0 + u < a.n) x[u][v] = ld_ro(a.p[k0 + u] + base + c);
      }
    }
    if (!kEarly && !kLateResidual && k0 + U >= a.n) load_residual();  // with the last partials
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float f[8];
        unpack16<T>(x[u][v], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[v][e] += f[e];
      }
    }
  }
  if constexpr (!kEarly) {
    // The same part of the rows one wave of CTAs ahead, on its way to L2.
    const int t = threadIdx.x;
    if (live && c1 > c0 && a.ahead > 0 && row + a.ahead < a.m && t <= a.n) {
      const uint32_t bytes = static_cast<uint32_t>(c1 - c0) * 16u;
      const int64_t at = base + a.ahead * a.P + c0;
      if (t < a.n)
        prefetch_l2(a.p[t] + at, bytes);
      else
        prefetch_l2(a.res + at * kParts, kParts * bytes);
    }
  }
  if (a.post != nullptr) {
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(acc[v][e], acc[v][e], ss);
    }
    if constexpr (!kEarly && !kLate) load(pw, a.post);
    const float total = row_sum(ss, nullptr, 0, q, S, sh, a);
    if constexpr (kLate) load(pw, a.post);
    const float inv = rsqrtf(total / a.H + a.eps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float f[8];
      unpack16<T>(pw[v], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[v][e] = (acc[v][e] * inv) * (f[e] + a.offset);
    }
  }
  if constexpr (kLateResidual) load_residual();
  if (gate != nullptr) {
    if constexpr (!kEarly) load(gv, gate);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float f[8];
      unpack16<T>(gv[v], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[v][e] *= f[e];
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = c0 + T0 + v * step;
    float f[8];
    unpack_residual<T, R32>(res[v], f);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[v][e] = fmaf(acc[v][e], a.block_scale, f[e] * a.residual_scale);
    if (c < end) {
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(acc[v][e], acc[v][e], ss);
      if constexpr (R32) {
        uint4 *to = a.rout + (base + c) * 2;
        const float(&y)[8] = acc[v];
        st_stream(to, make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]),
                                 __float_as_uint(y[3])));
        st_stream(to + 1, make_uint4(__float_as_uint(y[4]), __float_as_uint(y[5]), __float_as_uint(y[6]),
                                     __float_as_uint(y[7])));
      } else {
        st_stream(a.rout + base + c, pack16<T>(acc[v]));
      }
    }
  }
  if constexpr (!kEarly && !kLate) load(wv, a.w);
  if (a.scales == nullptr) {
    const float total = row_sum(ss, nullptr, 1, q, S, sh, a);
    if constexpr (kLate) load(wv, a.w);
    const float inv = rsqrtf(total / a.H + a.eps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = c0 + T0 + v * step;
      float f[8];
      unpack16<T>(wv[v], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = (acc[v][e] * inv) * (f[e] + a.offset);
      if (c < end) st_stream(static_cast<uint4 *>(a.out) + base + c, pack16<T>(f));
    }
    return;
  }
  // In bytes.  A row whose norm holds anything that is not finite gets zeros
  // and a scale of NaN.
  if constexpr (kLate) load(wv, a.w);
  if (!(ss < INFINITY)) {
    // Squares past fp32's end: the norm of finite values is 0, and their product
    // with the weight may pass the end too.
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[v][e] = 0.f * acc[v][e];
    }
  }
  uint32_t top = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = c0 + T0 + v * step;
    float f[8];
    unpack16<T>(wv[v], f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      acc[v][e] *= f[e] + a.offset;
      if (c < end) top = max(top, magnitude_bits(acc[v][e]));
    }
  }
  const float total = row_sum(ss, &top, 1, q, S, sh, a);
  const float inv = rsqrtf(total / a.H + a.eps);
  const float most = __uint_as_float(top);
  const float scale = most * inv / 127.f;
  const bool fine = top < kInfinityBits && magnitude_bits(scale) < kInfinityBits;
  // 2^100 keeps the quotient finite for rows of tiny values.
  const float up = most < 0x1p-100f ? 0x1p100f : 1.f;
  const bool some = fine && scale != 0.f;
  const float by = some ? 127.f / (most * up) : 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = c0 + T0 + v * step;
    float b[8];
    if (some && up == 1.f) {
#pragma unroll
      for (int e = 0; e < 8; ++e) b[e] = fmaf(acc[v][e], by, kRoundingBias);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) b[e] = fmaf(some ? acc[v][e] * up : 0.f, by, kRoundingBias);
    }
    if (c < end)
      __stcs(static_cast<uint2 *>(a.out) + base + c, make_uint2(bytes_of_biased(b[0], b[1], b[2], b[3]),
                                                               bytes_of_biased(b[4], b[5], b[6], b[7])));
  }
  if (live && q == 0 && threadIdx.x == 0) a.scales[row] = fine ? scale : __uint_as_float(0x7FC00000u);
}

using BlockNormKernel = void (*)(BlockNormArgs);

// A CTA a row with 2 or 4 packs a thread and at most 512 or 256 threads, or a
// cluster a row with 1 or 4 and at most 1024 or 256.  *registers: of a thread,
// at most.
BlockNormKernel block_norm_bf16(bool r32, bool cluster, int vpt, int *registers);
BlockNormKernel block_norm_f16(bool r32, bool cluster, int vpt, int *registers);

template <typename T, bool R32>
inline BlockNormKernel block_norm_rows(bool cluster, int vpt, int *registers) {
  *registers = vpt == 4 ? 80 : 64;
  if (cluster)
    return vpt == 1 ? &k_block_norm<T, R32, 1, 1024, 1, true> : &k_block_norm<T, R32, 4, 256, 3, true>;
  return vpt == 2 ? &k_block_norm<T, R32, 2, 512, 2, false> : &k_block_norm<T, R32, 4, 256, 3, false>;
}

template <typename T>
inline BlockNormKernel block_norm_of(bool r32, bool cluster, int vpt, int *registers) {
  return r32 ? block_norm_rows<T, true>(cluster, vpt, registers)
             : block_norm_rows<T, false>(cluster, vpt, registers);
}

}  // namespace arn
