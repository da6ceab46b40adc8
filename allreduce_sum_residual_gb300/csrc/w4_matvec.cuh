// Products of a few rows with 4-bit weights (ar_w4_matvec and
// ar_w4_matvec_experts): the kernel.
//
//   out[p, n] = sum_k x[p, k] (q[n, k] - z[n, k/G]) s[n, k/G]
//
// Bound by the weights' bytes: at 6.8 TB/s an SM has to take in some 47
// weights a clock, which leaves under three instruction slots for each --
// more than one row of fp32 multiply-adds would use up.  So the products run
// on mma.sync (m16n8k16, fp16, fp32 sums) with the weights as the 16-row
// operand and up to 8 NT rows of x as its columns: the arithmetic per weight
// is then the unpacking alone, whatever the number of columns.  (tcgen05
// would want the unpacked weights written back to shared memory, four times
// the bytes that came in; its rate is of no use to a kernel that reads each
// weight once.)
//
// Unpacking.  Logic operations run at half the rate of multiply-adds, so
// each word of eight weights costs one shift and four logic operations, one
// for each pair: four bits under the exponent of 1024 are the fp16 number
// 1024 + q, or 1024 + 16 q where they stand four bits higher.  One half2 add
// or multiply-add takes off the offset and the zero point.  All of it is
// exact: q - z is an integer in [-15, 15].  (bf16 has seven bits behind its
// leading one, room for one of the two places: eight integer operations a
// word instead of five, and 20 % more time where a batch of 32 tokens meets
// 112 experts' 1024 x 6144.)
//
// fp16 for x.  A column of x is scaled by the power of two that brings its
// largest finite magnitude to [2^13, 2^14), and its sums are scaled back.
// Every bf16 down to 2^-30 of the column's largest is then exact in fp16,
// smaller ones are rounded to a multiple of 2^-38 of it.  The tensor core
// sums a group's products in fp32, the group's scale multiplies that sum in
// fp32, and the groups are added in fp32: a warp's, then the warps' in
// order, CTA by CTA.
//
// Layout.  The weights are read as they are stored.  A warp takes units of
// 16 R rows x 128 k (64 bytes a row) into its own ring of shared memory with
// 16-byte asynchronous copies; nothing but the warp waits for it.  A lane
// (g, t) reads the words t, t + 4, ... of row g with groups of 32, so that
// all k of one product lie in one 32, two neighbouring words of each 64 with
// groups of 64, and four neighbouring words with groups of 128: one wide
// load where the group allows it.  The row stride (112, 96, 64 bytes) keeps
// each of these free of bank conflicts.  The pairs of a word come out as
// (i, i + 4), so x is stored with its eights in that order, in the order of
// the lanes.
//
// Work.  An item is 16 R rows x one column set (an expert's tokens, up to
// 8 NT).  A cluster of S CTAs takes a contiguous range of items, CTA q of it
// the units q, q + S, ... of each.  A CTA's warps form teams: a team takes
// items of the range in turn, and its warps the units of an item in turn.
// The ring runs on across items.
#pragma once

#include <cuda_fp16.h>

#include "experts.cuh"

namespace arn {

constexpr int kW4MaxWarps = 16;
constexpr int kW4UnitK = 128;  // k of a unit

struct W4Args {
  const uint4 *x;      // rows of K bf16
  const int32_t *ids;  // [pairs] experts; null: one matrix, every row of x
  const uint8_t *q;
  const uint8_t *scales;
  const uint8_t *zeros;
  __nv_bfloat16 *out;
  int64_t scale_count;  // scales, and zero points, of the whole array
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
  int team;         // warps of a team
  int xs_offset, red_offset, ids_offset;  // shared memory
  int smem_bytes;
  int *status;
};

// Units of a warp's ring: two to five in flight behind the one in use, 64 KB
// or more an SM with the plan's warps.
__host__ __device__ constexpr int w4_depth(int r) { return r == 1 ? 6 : 3; }
__host__ __device__ constexpr int w4_row_bytes(int group) {
  return group == 32 ? 112 : group == 64 ? 96 : 64;
}
// Scales and zero points of a row: behind its weights, or with groups of 128
// behind the unit's.
__host__ __device__ constexpr int w4_slot_bytes(int r, int group) {
  return 16 * r * (w4_row_bytes(group) + (group == 128 ? 8 : 0));
}

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

// d = A B, and d += A B.
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_next(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (word & mask) | bits in one operation, which two constants seldom become
// by themselves.
__device__ __forceinline__ uint32_t and_or(uint32_t word, uint32_t mask, uint32_t bits) {
  uint32_t v;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(word), "r"(mask), "r"(bits));
  return v;
}
// What comes off a pair: 1024 + z from one in the low bits, 64 + z from one
// four bits higher, once its 1024 + 16 q is divided by 16.
struct Offsets {
  uint32_t low, high;
};
__device__ __forceinline__ Offsets offsets_of(uint32_t z) {
  const uint32_t twice = z | z << 16;
  return Offsets{0xE400E400u | twice, 0xD400D400u | twice << 4};
}
__device__ __forceinline__ __half2 as_half2(uint32_t v) { return *reinterpret_cast<__half2 *>(&v); }
__device__ __forceinline__ uint32_t as_bits(__half2 v) { return *reinterpret_cast<uint32_t *>(&v); }
// Weights i and i + 4 of a word, i = 0 .. 3, less the zero point.
__device__ __forceinline__ void unpack_word(uint32_t (&p)[4], uint32_t word, const Offsets &o) {
  const __half2 sixteenth = as_half2(0x2C002C00u);
  const uint32_t next = word >> 8;
  p[0] = as_bits(__hadd2(as_half2(and_or(word, 0x000F000Fu, 0x64006400u)), as_half2(o.low)));
  p[1] = as_bits(__hfma2(as_half2(and_or(word, 0x00F000F0u, 0x64006400u)), sixteenth,
                         as_half2(o.high)));
  p[2] = as_bits(__hadd2(as_half2(and_or(next, 0x000F000Fu, 0x64006400u)), as_half2(o.low)));
  p[3] = as_bits(__hfma2(as_half2(and_or(next, 0x00F000F0u, 0x64006400u)), sixteenth,
                         as_half2(o.high)));
}

// Shared memory by its 32-bit addresses.
__device__ __forceinline__ uint4 lds_128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at));
  return v;
}
__device__ __forceinline__ uint2 lds_64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds_32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds_16(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds_8(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}

// Words 0 .. 3 of lane t of a row (the order of the steps).
template <int G>
__device__ __forceinline__ void load_words(uint32_t (&w)[4], uint32_t row, int t) {
  if constexpr (G == 128) {
    const uint4 v = lds_128(row + t * 16);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (G == 64) {
    const uint2 u = lds_64(row + t * 8), v = lds_64(row + 32 + t * 8);
    w[0] = u.x, w[1] = u.y, w[2] = v.x, w[3] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = lds_32(row + i * 16 + t * 4);
  }
}
// Where the eight k number k8 of a unit stand: step * 4 + lane.
template <int G>
__device__ __forceinline__ int step_lane(int k8) {
  if constexpr (G == 128) return (k8 & 3) * 4 + (k8 >> 2);
  if constexpr (G == 64) return ((k8 >> 3) * 2 + (k8 & 1)) * 4 + ((k8 >> 1) & 3);
  return k8;
}

// The power of two that a column whose largest finite magnitude has these
// fp32 bits is divided by; both it and its inverse are normal numbers.
__device__ __forceinline__ int exponent_of(int top) { return max((top >> 23) - 127 - 13, -126); }
// Two bf16 times a power of two, as fp16.
__device__ __forceinline__ uint32_t halves_of(uint32_t two, float scale) {
  return as_bits(__floats2half2_rn(__uint_as_float(two << 16) * scale,
                                   __uint_as_float(two & 0xFFFF0000u) * scale));
}

__device__ __forceinline__ void prefetch_line(const void *p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
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

// ST: AR_TYPE_* of the scales; ZEROS: whether there are zero points.
template <int R, int NT, int G, int ST, bool ZEROS, bool EXPERTS>
__global__ void __launch_bounds__(kW4MaxWarps * 32, 1) k_w4_matvec(const __grid_constant__ W4Args a) {
  extern __shared__ __align__(16) unsigned char w4_smem[];
  constexpr int kDepth = w4_depth(R), kSlot = w4_slot_bytes(R, G);
  constexpr int kRowBytes = w4_row_bytes(G);
  constexpr int kGroups = kW4UnitK / G;  // groups of a unit
  constexpr int kRows = 16 * R;
  // Of local row lr: its scale words at lr * kScaleStride + kScaleAt, its
  // zero points kZeroAt behind them.
  constexpr int kScaleAt = G == 128 ? kRows * 64 : 64;
  constexpr int kScaleStride = G == 128 ? 8 : kRowBytes;
  constexpr int kZeroAt = G == 128 ? 4 : G == 64 ? 8 : 32;
  constexpr int kScaleBytes = ST == AR_TYPE_F32 ? 4 : 2;
  // Aligned words that hold a unit's scales, or zero points, of one row.
  constexpr int kScaleWords = ST == AR_TYPE_F32 ? kGroups : kGroups == 1 ? 1 : kGroups / 2 + 1;
  constexpr int kZeroWords = kGroups == 1 ? 1 : 2;

  const int threads = blockDim.x, warps = threads >> 5;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int S = a.split;
  const int rank = S > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int cluster_id = static_cast<int>(blockIdx.x) / S, clusters = static_cast<int>(gridDim.x) / S;
  const int units = (a.units - rank + S - 1) / S;  // this CTA's units of an item
  const int teams = warps / a.team, team = warp / a.team, member = warp % a.team;
  const int64_t row_bytes = a.K / 2;

  unsigned char *ring = w4_smem + warp * (kDepth * kSlot);
  uint4 *xs = reinterpret_cast<uint4 *>(w4_smem + a.xs_offset);
  float *red = reinterpret_cast<float *>(w4_smem + a.red_offset);

  // Experts: ids16[p] the expert of pair p (-1: none), sets[e] the number of
  // column sets before expert e.
  int16_t *ids16 = reinterpret_cast<int16_t *>(w4_smem + a.ids_offset);
  __shared__ int sets[EXPERTS ? AR_MAX_EXPERTS + 1 : 1];
  __shared__ int col_pair[8 * NT];
  __shared__ int col_count;
  __shared__ int col_top[8 * NT];  // bits of a column's largest finite |x|
  __shared__ uint4 zero16;

  int nsets = (a.pairs + a.cols - 1) / a.cols;
  if constexpr (!EXPERTS) {
    // The first units' lines on their way to L2 while the previous grid
    // drains: nothing enters this SM before the wait.
    const int64_t total = static_cast<int64_t>(nsets) * a.row_blocks;
    const int64_t item = total * cluster_id / clusters + team;
    if (item < total * (cluster_id + 1) / clusters && (t & 1) == 0) {
      const int block = static_cast<int>(item % a.row_blocks);
      for (int d = 0, lu = member; d < kDepth - 1 && lu < units; ++d, lu += a.team) {
        const int64_t piece = static_cast<int64_t>(lu * S + rank) * 64 + t * 16;
#pragma unroll
        for (int i = 0; i < 2 * R; ++i)
          if (piece < row_bytes)
            prefetch_line(a.q + w4_row<R>(a, block, g + 8 * i) * row_bytes + piece);
      }
    }
  }
  pdl_wait_prior_grid();
  pdl_launch_dependents();

  if constexpr (EXPERTS) {
    for (int e = tid; e <= AR_MAX_EXPERTS; e += threads) sets[e] = 0;
    __syncthreads();
    for (int p = tid; p < a.pairs; p += threads) {
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
        for (int n = tid; n < a.width; n += threads)
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

  // The fetching side of the ring.  f_item: the team's item, f_base and
  // f_end: the column set's part of the range.
  int f_item = item0 + team, f_base = item0, f_end = item0, f_unit = member, f_slot = 0;
  int f_block0 = 0;              // block of f_base
  int64_t f_first = 0;           // first row of W of the set's expert
  const uint8_t *f_q = nullptr;  // this lane's 16 bytes of the expert's first row
  uint32_t f_off[2 * R];         // the rows' distances, in 16 bytes
  const uint8_t *f_s = nullptr, *f_z = nullptr;  // scales and zero points of row `lane`
  bool f_tail = false;           // near the end of their arrays
  const int full_units = static_cast<int>(row_bytes >> 6);  // units of a row that are whole
  auto next_item = [&]() {       // from f_item on, the team's first item that exists
    if (f_item >= f_end) {
      while (f_item >= f_end && f_end < item1) {
        f_base = f_end;
        f_item = f_base + team;
        const int set = f_base / a.row_blocks;
        f_block0 = f_base - set * a.row_blocks;
        f_end = min(item1, f_base - f_block0 + a.row_blocks);
        f_first = static_cast<int64_t>(expert_of(set)) * a.N;
      }
      if (f_item >= f_end) return;
      f_q = a.q + f_first * row_bytes + t * 16;
    }
    const int block = f_item - f_base + f_block0;
#pragma unroll
    for (int i = 0; i < 2 * R; ++i)
      f_off[i] = static_cast<uint32_t>(w4_row<R>(a, block, g + 8 * i)) *
                 static_cast<uint32_t>(row_bytes >> 4);
    const int64_t el = (f_first + w4_row<R>(a, block, lane & (kRows - 1))) * a.ng;
    f_s = a.scales + el * kScaleBytes;
    if constexpr (ZEROS) f_z = a.zeros + el;
    f_tail = el + a.ng + 16 > a.scale_count;
  };
  next_item();
  auto fetch = [&]() {
    while (f_item < f_end && f_unit >= units) {
      // The team's warps take up the next item where this one left them.
      f_unit -= units;
      f_item += teams;
      next_item();
    }
    if (f_item < f_end) {
      const int u = f_unit * S + rank;
      const uint32_t slot = smem_addr(ring) + f_slot * kSlot;
      const uint32_t to = slot + g * kRowBytes + t * 16;
      if (u < full_units) {
        const uint8_t *src = f_q + u * 64;
#pragma unroll
        for (int i = 0; i < 2 * R; ++i)
          cp_async_16(to + 8 * i * kRowBytes, src + static_cast<uint64_t>(f_off[i]) * 16, 16u);
      } else {  // the row ends inside the unit: zeros behind it
        const bool here = u * 64 + t * 16 < static_cast<int>(row_bytes);
        const uint8_t *src = f_q + (here ? u * 64 : 0);
#pragma unroll
        for (int i = 0; i < 2 * R; ++i)
          cp_async_16(to + 8 * i * kRowBytes, src + static_cast<uint64_t>(f_off[i]) * 16,
                      here ? 16u : 0u);
      }
      // The aligned words around the unit's scales and zero points, cut off
      // at the end of their arrays.
      if (lane < kRows) {
        const uint32_t to_s = slot + kScaleAt + lane * kScaleStride;
        auto words = [&](uint32_t dst, const uint8_t *p, const uint8_t *end, int n) {
          const uint8_t *w = reinterpret_cast<const uint8_t *>(reinterpret_cast<uintptr_t>(p) &
                                                               ~uintptr_t{3});
          if (!f_tail) {
#pragma unroll
            for (int i = 0; i < n; ++i) cp_async_4(dst + 4 * i, w + 4 * i, 4u);
          } else {
#pragma unroll
            for (int i = 0; i < n; ++i) {
              const int64_t left = end - (w + 4 * i);
              if (left > 0)
                cp_async_4(dst + 4 * i, w + 4 * i, left < 4 ? static_cast<uint32_t>(left) : 4u);
            }
          }
        };
        words(to_s, f_s + u * (kGroups * kScaleBytes), a.scales + a.scale_count * kScaleBytes,
              kScaleWords);
        if constexpr (ZEROS)
          words(to_s + kZeroAt, f_z + u * kGroups, a.zeros + a.scale_count, kZeroWords);
      }
      f_slot = f_slot + 1 == kDepth ? 0 : f_slot + 1;
      f_unit += a.team;
    }
    cp_async_commit();  // an empty group at the end keeps the count
  };
#pragma unroll 1
  for (int i = 0; i < kDepth - 1; ++i) fetch();

  const bool act = a.act == AR_ACT_SILU_MUL;
  const int outs = act ? 8 * R : kRows;  // outputs of an item's column
  int c_unit = member, slot_at = 0, parity = 0;
#pragma unroll 1
  for (int seg = item0; seg < item1;) {
    // The part of the range that has one column set.
    const int set = seg / a.row_blocks;
    const int seg_end = min(item1, (set + 1) * a.row_blocks);
    const int expert = expert_of(set);
    __syncthreads();  // nobody uses the last set's x any more
    if (tid == 0) zero16 = make_uint4(0, 0, 0, 0);
    if (tid < 8 * NT) col_top[tid] = 0;
    if constexpr (EXPERTS) {
      if (warp == 0) {  // the set's columns, in the order of the pairs
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
      const int n = min(a.cols, a.pairs - set * a.cols);
      if (tid < n) col_pair[tid] = set * a.cols + tid;
      if (tid == 0) col_count = n;
    }
    __syncthreads();
    const int ncols = col_count;
    {
      const int pieces = units * 16;  // eights of a column
      auto place = [&](int i, int *col) -> uint4 * {  // of eight i of all columns
        *col = i / pieces;
        const int j = i - *col * pieces, to = step_lane<G>(j & 15);
        return xs + (((j >> 4) * 4 + (to >> 2)) * a.cols + *col) * 4 + (to & 3);
      };
      for (int i0 = 0; i0 < pieces * ncols; i0 += threads) {
        // Sixteen lanes hold eights of one column.
        const int i = i0 + tid;
        int col, top = 0;
        uint4 *to = place(i, &col);
        if (col < ncols) {
          const int j = i - col * pieces, at = ((j >> 4) * S + rank) * 16 + (j & 15);
          uint4 w = make_uint4(0, 0, 0, 0);
          if (at * 8 < a.K)
            w = __ldg(a.x + static_cast<int64_t>(col_pair[col] / a.k) * (a.K / 8) + at);
          float f[8];
          unpack8(w, f);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int bits = __float_as_int(f[e]) & 0x7FFFFFFF;
            if (bits < 0x7F800000 && bits > top) top = bits;
          }
          *to = make_uint4(__byte_perm(w.x, w.z, 0x5410), __byte_perm(w.x, w.z, 0x7632),
                           __byte_perm(w.y, w.w, 0x5410), __byte_perm(w.y, w.w, 0x7632));
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        if ((lane & 15) == 0 && col < ncols && top > 0) atomicMax(&col_top[col], top);
      }
      __syncthreads();
      for (int i = tid; i < pieces * ncols; i += threads) {  // what this thread has put there
        int col;
        uint4 *to = place(i, &col);
        const float down = __int_as_float((127 - exponent_of(col_top[col])) << 23);
        uint4 v = *to;
        v.x = halves_of(v.x, down), v.y = halves_of(v.y, down);
        v.z = halves_of(v.z, down), v.w = halves_of(v.w, down);
        *to = v;
      }
    }
    __syncthreads();

    // This lane's eights of x: column g of each tile, or zeros.  And where
    // its two columns of each tile's sums go.
    uint32_t xp[NT], xstep[NT];
    __nv_bfloat16 *op[NT][2];
    float up[NT][2];  // the columns' powers of two
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const bool in = n * 8 + g < ncols;
      xp[n] = in ? smem_addr(xs + (n * 8 + g) * 4 + t) : smem_addr(&zero16);
      xstep[n] = in ? a.cols * 64 : 0;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = n * 8 + 2 * t + c;
        up[n][c] = __int_as_float((127 + exponent_of(col_top[col])) << 23);
        op[n][c] = col < ncols ? a.out + static_cast<int64_t>(col_pair[col]) * a.width : nullptr;
      }
    }
    const int rounds = (seg_end - seg + teams - 1) / teams;
#pragma unroll 1
    for (int round = 0; round < rounds; ++round) {
      const int item = seg + round * teams + team;
      const bool has = item < seg_end;
      const int block = item - set * a.row_blocks;
      float acc[R][NT][4];
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[r][n][c] = 0.f;
      if (has) {
        int el_low[R][2];  // low bits of the rows' first group numbers
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            el_low[r][h] =
                ((expert * a.N + w4_row<R>(a, block, r * 16 + h * 8 + g)) & 3) * (a.ng & 3);
#pragma unroll 1
        for (; c_unit < units; c_unit += a.team) {
          cp_async_wait<kDepth - 2>();
          __syncwarp();  // every lane's copies are here, and the slot before is free
          fetch();
          const uint32_t slot = smem_addr(ring) + slot_at * kSlot;
          slot_at = slot_at + 1 == kDepth ? 0 : slot_at + 1;
          uint4 b[4][NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint32_t p = xp[n] + c_unit * 4 * xstep[n];
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i][n] = lds_128(p + i * xstep[n]);
          }
          const int u0 = (c_unit * S + rank) * kGroups;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const uint32_t row = slot + (r * 16 + g) * kRowBytes;
            uint32_t w0[4], w1[4];
            load_words<G>(w0, row, t);
            load_words<G>(w1, row + 8 * kRowBytes, t);
            const uint32_t sc = slot + kScaleAt + (r * 16 + g) * kScaleStride;
#pragma unroll
            for (int gi = 0; gi < kGroups; ++gi) {
              // Scale and zero point of the two rows' group.
              float s[2];
              Offsets o[2];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t p = sc + h * 8 * kScaleStride;
                const int low = el_low[r][h] + u0;
                if constexpr (ST == AR_TYPE_F32) {
                  s[h] = __uint_as_float(lds_32(p + gi * 4));
                } else {
                  const uint32_t v = lds_16(p + ((low & 1) + gi) * 2);
                  s[h] = ST == AR_TYPE_BF16
                             ? __uint_as_float(v << 16)
                             : __half2float(__ushort_as_half(static_cast<unsigned short>(v)));
                }
                // Behind the row's end stands another row's scale.
                if (kGroups > 1 && u0 + gi >= a.ng) s[h] = 0.f;
                o[h] = offsets_of(ZEROS ? lds_8(p + kZeroAt + (low & 3) + gi) & 15u : 8u);
              }
              float d[NT][4];
              constexpr int kSteps = 4 / kGroups;
#pragma unroll
              for (int i = gi * kSteps; i < (gi + 1) * kSteps; ++i) {
                uint32_t p[4], q[4];
                unpack_word(p, w0[i], o[0]);
                unpack_word(q, w1[i], o[1]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  if (i == gi * kSteps) mma_first(d[n], p[0], q[0], p[1], q[1], b[i][n].x, b[i][n].y);
                  else mma_next(d[n], p[0], q[0], p[1], q[1], b[i][n].x, b[i][n].y);
                  mma_next(d[n], p[2], q[2], p[3], q[3], b[i][n].z, b[i][n].w);
                }
              }
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[r][n][c] = fmaf(s[c >> 1], d[n][c], acc[r][n][c]);
            }
          }
        }
        c_unit -= units;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[r][n][c] *= up[n][c & 1];
      }

      if (a.team == 1 && S == 1) {  // the warp has the whole sums
        if (has) {
          const int o0 = block * outs + g;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              __nv_bfloat16 *p = op[n][c] + o0;
              if (op[n][c] == nullptr) continue;
#pragma unroll
              for (int r = 0; r < R; ++r) {
                if (act) {
                  if (o0 + r * 8 < a.width)
                    p[r * 8] = __float2bfloat16_rn(gated(acc[r][n][c], acc[r][n][c + 2]));
                } else {
                  if (o0 + r * 16 < a.width) p[r * 16] = __float2bfloat16_rn(acc[r][n][c]);
                  if (o0 + r * 16 + 8 < a.width) p[r * 16 + 8] = __float2bfloat16_rn(acc[r][n][c + 2]);
                }
              }
            }
        }
        continue;
      }
      // The warps' sums: red[parity][warp][column][row].  A buffer is written
      // again two items on, behind a barrier that every reader has passed.
      const int stride = a.cols * kRows;
      float *buf = red + (parity * warps + team * a.team) * stride;
      parity ^= 1;
      if (has) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int col = n * 8 + 2 * t + (c & 1), row = r * 16 + (c >> 1) * 8 + g;
              if (col < ncols) buf[member * stride + col * kRows + row] = acc[r][n][c];
            }
      }
      if (S > 1) {
        __syncwarp();
        cluster_arrive_release();
        cluster_wait_acquire();
      } else if (has) {
        asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(a.team * 32) : "memory");
      }
      if (has) {
        auto sum_of = [&](int col, int row) -> float {
          float v = 0.f;
          const float *p = buf + col * kRows + row;
          if (S == 1) {
            for (int w = 0; w < a.team; ++w) v += p[w * stride];
          } else {
            for (int c = 0; c < S; ++c)
              for (int w = 0; w < a.team; ++w) v += ld_cluster_f32(p + w * stride, c);
          }
          return v;
        };
        for (int i = (member * 32 + lane) * S + rank; i < ncols * outs; i += a.team * 32 * S) {
          const int col = i / outs, o = i - col * outs;
          const int row = act ? (o >> 3) * 16 + (o & 7) : o;
          float v = sum_of(col, row);
          if (act) v = gated(v, sum_of(col, row + 8));
          if (block * outs + o < a.width)
            a.out[static_cast<int64_t>(col_pair[col]) * a.width + block * outs + o] =
                __float2bfloat16_rn(v);
        }
      }
    }
    seg = seg_end;
  }
  cp_async_wait<0>();
  if (S > 1) {  // no CTA leaves while another reads its sums
    __syncwarp();
    cluster_arrive_release();
    cluster_wait_acquire();
  }
}

using W4Kernel = void (*)(W4Args);
template <int ST, bool ZEROS, bool EXPERTS, int R, int NT>
inline W4Kernel w4_pick_group(int group) {
  return group == 32 ? &k_w4_matvec<R, NT, 32, ST, ZEROS, EXPERTS>
         : group == 64 ? &k_w4_matvec<R, NT, 64, ST, ZEROS, EXPERTS>
                       : &k_w4_matvec<R, NT, 128, ST, ZEROS, EXPERTS>;
}
template <int ST, bool ZEROS, bool EXPERTS>
inline W4Kernel w4_pick_tile(int r, int nt, int group) {
  if (nt == 1)
    return r == 1 ? w4_pick_group<ST, ZEROS, EXPERTS, 1, 1>(group)
                  : w4_pick_group<ST, ZEROS, EXPERTS, 2, 1>(group);
  return r == 1 ? w4_pick_group<ST, ZEROS, EXPERTS, 1, 2>(group)
                : w4_pick_group<ST, ZEROS, EXPERTS, 2, 2>(group);
}

}  // namespace arn
