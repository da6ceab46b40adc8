// Products of a few rows with 4-bit weights (ar_w4_matvec and
// ar_w4_matvec_experts): the kernel.
//
//   out[p, n] = sum_k x[p, k] (q[n, k] - z[n, k/G]) s[n, k/G]
//
// Bound by the weights' bytes: at 6.8 TB/s an SM has to take in some 47
// weights a clock, which leaves under three instruction slots for each --
// more than one row of fp32 multiply-adds would use up.  So the products run
// on mma.sync (m16n8k16, bf16, fp32 sums) with the weights as the 16-row
// operand and up to 8 NT rows of x as its columns: the arithmetic per weight
// is then the unpacking alone, whatever the number of columns.  (tcgen05
// would want the unpacked weights written back to shared memory, four times
// the bytes that came in; its rate is of no use to a kernel that reads each
// weight once.)
//
// Exactness.  q - z is an integer in [-15, 15], exact in bf16: the four bits
// under the exponent of 128 are the number 128 + q, and 128 + z is
// subtracted from it.  The tensor core sums a group's products in fp32, the
// group's scale multiplies that sum in fp32, and the groups are added in
// fp32: first a warp's, then the warps' in order, then the CTAs' in order.
//
// Layout.  The weights are read as they are stored.  A warp takes units of
// 16 R rows x 128 k (64 bytes a row) into its own ring of shared memory with
// 16-byte asynchronous copies; nothing but the warp waits for it.  Rows lie
// 80 bytes apart (112 with groups of 32), so that the 32 words of an operand
// load fall into 32 banks; the bytes between hold the unit's scales and zero
// points.  Word t of a 16-byte piece of row g is lane (g, t)'s: its eight
// weights are two pairs for each of two products.  The pairs of a word come
// out as (i, i + 4), so x is stored with its eights in that order, once per
// column set.  Within one product all k belong to the same 32, so that every
// group size can be scaled after it.
//
// Work.  An item is 16 R rows x one column set (an expert's tokens, up to
// 8 NT).  A cluster of S CTAs takes a contiguous range of items, CTA q of it
// the units q, q + S, ... of each; the warps of a CTA take its units in
// turn.  The ring runs on across items.
#pragma once

#include <cuda_fp16.h>

#include "experts.cuh"

namespace arn {

constexpr int kW4Warps = 8;
constexpr int kW4Threads = kW4Warps * 32;
constexpr int kW4UnitK = 128;  // k of a unit

struct W4Args {
  const uint4 *x;      // rows of K bf16
  const int32_t *ids;  // [pairs] experts; null: one matrix, every row of x
  const uint8_t *q;
  const uint8_t *scales;
  const uint8_t *zeros;
  __nv_bfloat16 *out;
  int64_t scale_bytes, zero_bytes;  // of the whole arrays
  int pairs;        // rows of out
  int k;            // pair p takes row p / k of x
  int E, N, K, ng;  // ng: groups of a row
  int width;        // columns of out: N, or N / 2 with the gated activation
  int act;
  int scale_type;
  int units;        // units of a row: ceil(K / 128)
  int row_blocks;   // items of a column set
  int cols;         // most columns of a set
  int split;        // CTAs of a cluster
  int xs_offset, red_offset, part_offset, ids_offset;  // shared memory
  int smem_bytes;
  int *status;
};

template <int R>
__host__ __device__ constexpr int w4_depth() {  // units of a warp's ring
  return R == 1 ? 8 : R == 2 ? 5 : 3;
}
__host__ __device__ constexpr int w4_row_bytes(int group) { return group == 32 ? 112 : 80; }
__host__ __device__ constexpr int w4_zero_offset(int group) { return group == 32 ? 96 : 72; }

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Weights I and I + 4 of a word, minus the zero point: exact in bf16.
// `minus` holds 128 + z twice.
template <int I>
__device__ __forceinline__ uint32_t weight_pair(uint32_t word, uint32_t minus) {
  const uint32_t v = ((word >> (4 * I)) & 0x000F000Fu) | 0x43004300u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v),
                                   *reinterpret_cast<const __nv_bfloat162 *>(&minus));
  return *reinterpret_cast<const uint32_t *>(&d);
}

__device__ __forceinline__ float ld_cluster_f32(const float *local, uint32_t rank) {
  uint32_t at;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(local)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ float gated(float gate, float up) {
  return gate / (1.f + expf(-gate)) * up;
}

// Row of W behind local row lr of block b.  Local rows come in sixteens;
// with the gated activation the first eight are gate rows and the last eight
// the up rows of the same outputs.  Beyond the end: the last row, whose
// result is not stored.
template <int R>
__device__ __forceinline__ int w4_row(const W4Args &a, int block, int lr) {
  if (a.act == AR_ACT_SILU_MUL) {
    const int o = block * 8 * R + (lr >> 4) * 8 + (lr & 7);
    return min(o, a.width - 1) + ((lr >> 3) & 1) * a.width;
  }
  return min(block * 16 * R + lr, a.N - 1);
}

template <int R, int NT, int G, bool EXPERTS>
__global__ void __launch_bounds__(kW4Threads) k_w4_matvec(const __grid_constant__ W4Args a) {
  extern __shared__ __align__(16) unsigned char w4_smem[];
  constexpr int kDepth = w4_depth<R>();
  constexpr int kRowBytes = w4_row_bytes(G), kZeroOffset = w4_zero_offset(G);
  constexpr int kSlot = 16 * R * kRowBytes;
  constexpr int kGroups = kW4UnitK / G;  // groups of a unit
  constexpr int kRows = 16 * R;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int S = a.split;
  const int rank = S > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int cluster_id = static_cast<int>(blockIdx.x) / S, clusters = static_cast<int>(gridDim.x) / S;
  const int units = (a.units - rank + S - 1) / S;  // this CTA's units of an item

  unsigned char *ring = w4_smem + warp * (kDepth * kSlot);
  uint4 *xs = reinterpret_cast<uint4 *>(w4_smem + a.xs_offset);
  float *red = reinterpret_cast<float *>(w4_smem + a.red_offset);
  float *part = reinterpret_cast<float *>(w4_smem + a.part_offset);

  // Experts: ids16[p] the expert of pair p (-1: none), sets[e] the number of
  // column sets before expert e.
  int16_t *ids16 = reinterpret_cast<int16_t *>(w4_smem + a.ids_offset);
  __shared__ int sets[AR_MAX_EXPERTS + 1];
  __shared__ int col_pair[8 * NT];
  __shared__ int col_count;

  pdl_wait_prior_grid();
  pdl_launch_dependents();

  int nsets = (a.pairs + a.cols - 1) / a.cols;
  if constexpr (EXPERTS) {
    for (int e = tid; e <= AR_MAX_EXPERTS; e += kW4Threads) sets[e] = 0;
    __syncthreads();
    for (int p = tid; p < a.pairs; p += kW4Threads) {
      const int e = __ldg(a.ids + p);
      const bool ok = e >= 0 && e < a.E;
      ids16[p] = static_cast<int16_t>(ok ? e : -1);
      if (ok) atomicAdd(&sets[e], 1);
    }
    __syncthreads();
    if (warp == 0) {  // counts -> column sets before each expert
      constexpr int kEach = AR_MAX_EXPERTS / 32;
      int mine = 0;
      for (int i = 0; i < kEach; ++i) mine += (sets[lane * kEach + i] + a.cols - 1) / a.cols;
      int before = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, before, o);
        if (lane >= o) before += v;
      }
      if (lane == 31) sets[AR_MAX_EXPERTS] = before;
      before -= mine;
      for (int i = 0; i < kEach; ++i) {
        const int n = (sets[lane * kEach + i] + a.cols - 1) / a.cols;
        sets[lane * kEach + i] = before;
        before += n;
      }
    }
    __syncthreads();
    nsets = sets[AR_MAX_EXPERTS];
    // Pairs without an expert here: zero rows, spread over the grid.
    for (int p = blockIdx.x; p < a.pairs; p += gridDim.x)
      if (ids16[p] < 0)
        for (int n = tid; n < a.width; n += kW4Threads)
          a.out[static_cast<int64_t>(p) * a.width + n] = __float2bfloat16_rn(0.f);
  }
  const int64_t total = static_cast<int64_t>(nsets) * a.row_blocks;
  const int item0 = static_cast<int>(total * cluster_id / clusters);
  const int item1 = static_cast<int>(total * (cluster_id + 1) / clusters);

  // The expert of a column set.
  auto expert_of = [&](int set) -> int {
    if constexpr (!EXPERTS) return 0;
    int lo = 0, hi = AR_MAX_EXPERTS;  // sets[lo] <= set < sets[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sets[mid] <= set) lo = mid;
      else hi = mid;
    }
    return lo;
  };

  // Issue side of the ring: the next unit to fetch.
  int f_item = item0, f_unit = warp, f_slot = 0;
  int f_set = -1, f_block = 0;
  int64_t f_expert_row = 0;  // first row of W of the item's expert
  const int64_t row_bytes = a.K / 2;
  auto fetch = [&]() {
    if (f_item < item1 && f_unit < units) {
      const int set = f_item / a.row_blocks;
      if (set != f_set) {
        f_set = set;
        f_expert_row = static_cast<int64_t>(expert_of(set)) * a.N;
      }
      f_block = f_item - set * a.row_blocks;
      const int u = f_unit * S + rank;
      const uint32_t slot = smem_addr(ring + f_slot * kSlot);
      const int piece = u * 64 + t * 16;  // byte of the row
      const uint32_t bytes = piece < row_bytes ? 16u : 0u;
#pragma unroll
      for (int i = 0; i < 2 * R; ++i) {
        const int lr = g + 8 * i;
        const int64_t row = f_expert_row + w4_row<R>(a, f_block, lr);
        cp_async_16(slot + lr * kRowBytes + t * 16, a.q + row * row_bytes + (bytes ? piece : 0),
                    bytes);
      }
      // The aligned words around the unit's scales and zero points.
      const int size_log2 = a.scale_type == AR_TYPE_F32 ? 2 : 1;
#pragma unroll
      for (int i = 0; i < (kRows + 31) / 32; ++i) {
        const int lr = lane + 32 * i;
        if (lr < kRows) {
          const int64_t row = f_expert_row + w4_row<R>(a, f_block, lr);
          const int64_t el = row * a.ng + u * kGroups;
          const int64_t sb = (el << size_log2) & ~int64_t{3};
          const int words = a.scale_type == AR_TYPE_F32 ? kGroups : kGroups == 1 ? 1 : kGroups / 2 + 1;
          for (int w = 0; w < words; ++w) {
            const int64_t left = a.scale_bytes - (sb + 4 * w);
            const uint32_t n = left >= 4 ? 4u : left > 0 ? static_cast<uint32_t>(left) : 0u;
            cp_async_4(slot + lr * kRowBytes + 64 + 4 * w, a.scales + (n ? sb + 4 * w : 0), n);
          }
          if (a.zeros != nullptr) {
            const int64_t zb = el & ~int64_t{3};
#pragma unroll
            for (int w = 0; w < (kGroups == 1 ? 1 : 2); ++w) {
              const int64_t left = a.zero_bytes - (zb + 4 * w);
              const uint32_t n = left >= 4 ? 4u : left > 0 ? static_cast<uint32_t>(left) : 0u;
              cp_async_4(slot + lr * kRowBytes + kZeroOffset + 4 * w, a.zeros + (n ? zb + 4 * w : 0),
                         n);
            }
          }
        }
      }
      f_slot = f_slot + 1 == kDepth ? 0 : f_slot + 1;
      f_unit += kW4Warps;
      if (f_unit >= units) {
        f_unit = warp;
        ++f_item;
      }
    }
    cp_async_commit();  // an empty group at the end keeps the count
  };
#pragma unroll 1
  for (int i = 0; i < kDepth - 1; ++i) fetch();

  int slot_at = 0, staged = -1, ncols = 0, parity = 0;
#pragma unroll 1
  for (int item = item0; item < item1; ++item) {
    const int set = item / a.row_blocks, block = item - set * a.row_blocks;
    const int expert = expert_of(set);
    if (set != staged) {
      // The set's columns, in the order of the pairs, then their x.
      staged = set;
      __syncthreads();
      if constexpr (EXPERTS) {
        if (warp == 0) {
          const int skip = (set - sets[expert]) * a.cols;
          int seen = 0;
          for (int p0 = 0; p0 < a.pairs && seen < skip + a.cols; p0 += 32) {
            const bool is = p0 + lane < a.pairs && ids16[p0 + lane] == expert;
            const uint32_t who = __ballot_sync(0xFFFFFFFFu, is);
            const int at = seen + __popc(who & ((1u << lane) - 1u)) - skip;
            if (is && at >= 0 && at < a.cols) col_pair[at] = p0 + lane;
            seen += __popc(who);
          }
          if (lane == 0) col_count = min(seen - skip, a.cols);
        }
      } else {
        if (tid < min(a.cols, a.pairs - set * a.cols)) col_pair[tid] = set * a.cols + tid;
        if (tid == 0) col_count = min(a.cols, a.pairs - set * a.cols);
      }
      __syncthreads();
      ncols = col_count;
      const int pieces = units * 16;
      for (int i = tid; i < pieces * ncols; i += kW4Threads) {
        const int col = i / pieces, j = i - col * pieces;  // j: (unit, 32, eight)
        const int k8 = ((j >> 4) * S + rank) * 16 + (j & 15);  // eight of the row
        uint4 v = make_uint4(0, 0, 0, 0);
        if (k8 * 8 < a.K) {
          const int64_t row = col_pair[col] / a.k;
          const uint4 w = __ldg(a.x + row * (a.K / 8) + k8);
          v = make_uint4(__byte_perm(w.x, w.z, 0x5410), __byte_perm(w.x, w.z, 0x7632),
                         __byte_perm(w.y, w.w, 0x5410), __byte_perm(w.y, w.w, 0x7632));
        }
        xs[((j >> 2) * a.cols + col) * 4 + (j & 3)] = v;
      }
      __syncthreads();
    }

    float acc[R][NT][4];
    int el_low[R][2];  // low bits of the rows' first group number
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        el_low[r][h] = static_cast<int>(
            ((static_cast<int64_t>(expert) * a.N + w4_row<R>(a, block, r * 16 + h * 8 + g)) * a.ng) & 3);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[r][n][c] = 0.f;
    }
#pragma unroll 1
    for (int lu = warp; lu < units; lu += kW4Warps) {
      cp_async_wait<kDepth - 2>();
      __syncwarp();  // every lane's copies are here, and the slot before is free
      fetch();
      const unsigned char *slot = ring + slot_at * kSlot;
      slot_at = slot_at + 1 == kDepth ? 0 : slot_at + 1;
      const int u0 = (lu * S + rank) * kGroups;
      float d[R][NT][4];
      float s[R][2];
      uint32_t minus[R][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        constexpr int kPer = G / 32;  // 32s of a group
        const int gi = i / kPer;
        if (i % kPer == 0) {
#pragma unroll
          for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const unsigned char *row = slot + (r * 16 + h * 8 + g) * kRowBytes;
              const int low = (el_low[r][h] + u0) & 3;
              if (a.scale_type == AR_TYPE_F32) {
                s[r][h] = *reinterpret_cast<const float *>(row + 64 + gi * 4);
              } else {
                const uint16_t b =
                    *reinterpret_cast<const uint16_t *>(row + 64 + ((low & 1) + gi) * 2);
                s[r][h] = a.scale_type == AR_TYPE_BF16
                              ? __uint_as_float(static_cast<uint32_t>(b) << 16)
                              : __half2float(__ushort_as_half(b));
              }
              if (u0 + gi >= a.ng) s[r][h] = 0.f;  // behind the row: another row's scale
              const uint32_t z = a.zeros != nullptr ? row[kZeroOffset + low + gi] & 15u : 8u;
              minus[r][h] = 0x43004300u | z | (z << 16);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int c = 0; c < 4; ++c) d[r][n][c] = 0.f;
          }
        }
        uint4 b[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          b[n] = make_uint4(0, 0, 0, 0);
          if (n * 8 + g < ncols) b[n] = xs[((lu * 4 + i) * a.cols + n * 8 + g) * 4 + t];
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const unsigned char *at = slot + (r * 16 + g) * kRowBytes + i * 16 + t * 4;
          const uint32_t w0 = *reinterpret_cast<const uint32_t *>(at);
          const uint32_t w1 = *reinterpret_cast<const uint32_t *>(at + 8 * kRowBytes);
          const uint32_t p0 = weight_pair<0>(w0, minus[r][0]), p1 = weight_pair<0>(w1, minus[r][1]);
          const uint32_t p2 = weight_pair<1>(w0, minus[r][0]), p3 = weight_pair<1>(w1, minus[r][1]);
          const uint32_t p4 = weight_pair<2>(w0, minus[r][0]), p5 = weight_pair<2>(w1, minus[r][1]);
          const uint32_t p6 = weight_pair<3>(w0, minus[r][0]), p7 = weight_pair<3>(w1, minus[r][1]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_bf16(d[r][n], p0, p1, p2, p3, b[n].x, b[n].y);
            mma_bf16(d[r][n], p4, p5, p6, p7, b[n].z, b[n].w);
          }
        }
        if (i % kPer == kPer - 1) {
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int c = 0; c < 4; ++c) acc[r][n][c] = fmaf(s[r][c >> 1], d[r][n][c], acc[r][n][c]);
        }
      }
    }

    // The warps' sums, in order: red[warp][column][row].
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int col = n * 8 + 2 * t + (c & 1), row = r * 16 + (c >> 1) * 8 + g;
          if (col < ncols) red[(warp * a.cols + col) * kRows + row] = acc[r][n][c];
        }
    __syncthreads();
    const int warp_stride = a.cols * kRows;
    auto cta_sum = [&](int col, int row) -> float {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kW4Warps; ++w) v += red[w * warp_stride + col * kRows + row];
      return v;
    };
    float *mine = part + parity * warp_stride;
    if (S > 1) {
      for (int i = tid; i < ncols * kRows; i += kW4Threads) mine[i] = cta_sum(i / kRows, i % kRows);
      __syncwarp();
      // Double-buffered: a buffer is written again two items on, after a
      // barrier that every CTA reaches only behind its reads of it.
      cluster_arrive_release();
      cluster_wait_acquire();
      parity ^= 1;
    }
    auto item_sum = [&](int col, int row) -> float {
      if (S == 1) return cta_sum(col, row);
      float v = 0.f;
      for (int c = 0; c < S; ++c) v += ld_cluster_f32(mine + col * kRows + row, c);
      return v;
    };
    const bool act = a.act == AR_ACT_SILU_MUL;
    const int outs = act ? 8 * R : kRows;  // outputs of an item's column
    for (int i = tid * S + rank; i < ncols * outs; i += kW4Threads * S) {
      const int col = i / outs, o = i % outs;
      const int n = block * outs + o;
      if (n >= a.width) continue;
      float v;
      if (act) {
        const int row = (o >> 3) * 16 + (o & 7);
        v = gated(item_sum(col, row), item_sum(col, row + 8));
      } else {
        v = item_sum(col, o);
      }
      a.out[static_cast<int64_t>(col_pair[col]) * a.width + n] = __float2bfloat16_rn(v);
    }
    __syncthreads();  // red, and col_pair before the next set
  }
  cp_async_wait<0>();
  if (S > 1) {  // no CTA leaves while another reads its sums
    cluster_arrive_release();
    cluster_wait_acquire();
  }
}

using W4Kernel = void (*)(W4Args);
// [row tiles 1, 2, 4][column tiles 1, 2][group 32, 64, 128]
W4Kernel w4_dense_kernel(int r, int nt, int group);
W4Kernel w4_experts_kernel(int r, int nt, int group);

template <bool EXPERTS, int R, int NT>
inline W4Kernel w4_pick_group(int group) {
  return group == 32 ? &k_w4_matvec<R, NT, 32, EXPERTS>
         : group == 64 ? &k_w4_matvec<R, NT, 64, EXPERTS>
                       : &k_w4_matvec<R, NT, 128, EXPERTS>;
}
template <bool EXPERTS>
inline W4Kernel w4_pick(int r, int nt, int group) {
  if (nt == 1)
    return r == 1 ? w4_pick_group<EXPERTS, 1, 1>(group)
           : r == 2 ? w4_pick_group<EXPERTS, 2, 1>(group)
                    : w4_pick_group<EXPERTS, 4, 1>(group);
  return r == 1 ? w4_pick_group<EXPERTS, 1, 2>(group)
         : r == 2 ? w4_pick_group<EXPERTS, 2, 2>(group)
                  : w4_pick_group<EXPERTS, 4, 2>(group);
}

}  // namespace arn
