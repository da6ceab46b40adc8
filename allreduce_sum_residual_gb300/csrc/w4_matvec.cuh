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
// or multiply-add takes off the offset and the zero point (a published
// method: Kim, Henry, Fahim and Awadalla, "Who Says Elephants Can't Run",
// 2022).  All of it is exact: q - z is an integer in [-15, 15].  (bf16 has
// seven bits behind its leading one, room for one of the two places: eight
// integer operations a word instead of five, and 20 % more time where a batch
// of 32 tokens meets 112 experts' 1024 x 6144.)
//
// fp16 for x.  A column of x is scaled by the power of two that brings its
// largest finite magnitude to [2^13, 2^14), and its sums are scaled back.
// Every bf16 down to 2^-30 of the column's largest is then exact in fp16,
// smaller ones are rounded to a multiple of 2^-38 of it.  The tensor core
// sums a group's products in fp32, the group's scale multiplies that sum in
// fp32, and the groups are added in fp32: a warp's, then those of the team's
// warps in order, then the phases'.  (What passes fp32's end on the way,
// with scales of 2^95 and more, is computed again behind the items.)
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
// the lanes.  (One warp that feeds all rings by tensor-map copies was
// measured and dropped: 70 ns a 2 KB box, where memory brings one in 45.)
//
// Work.  An item is 16 R rows x one column set (an expert's tokens, up to
// 8 NT).  A CTA takes a contiguous range of items, its warps form teams, a
// team takes items of the range in turn, and its warps the units of the
// team's items in turn, whatever item they belong to: all warps do the same
// number of units, and the ring runs on across items.  A warp that ends an
// item leaves its sums in shared memory, goes on, and adds up its part of
// the item before once every warp of the team has left that one (mbarriers,
// bounded waits); a team of one needs none of this.  x of as many column
// sets as fit is unpacked into shared memory at once.  Where not even one
// set fits, the range is walked in phases, a part of K in each, and the sums
// so far wait in shared memory.
#pragma once

#include <cuda_fp16.h>

#include "experts.cuh"

namespace arn {

constexpr int kW4MaxWarps = 16;  // four a scheduler, 128 registers a thread
constexpr int kW4PartK = 128;  // k of a unit's part
// Parts of a unit.  Two where one row tile and one column tile leave little
// to do for a unit's fixed work (one row, 7168 x 7168: 10.8 us, one part 6 % more);
// not with two column tiles or groups of 32, whose x or scales need the room.
__host__ __device__ constexpr int w4_parts(int r, int nt, int group) {
  return r == 1 && nt == 1 && group != 32 ? 2 : 1;
}

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
  int first;        // number of q's first expert
  int E, N, K, ng;  // ng: groups of a row
  int width;        // columns of out: N, or N / 2 with the gated activation
  int act;
  int units;        // units of a row: ceil(K / (128 parts))
  int row_blocks;   // items of a column set
  int cols;         // most columns of a set
  int x_cols;       // columns of x that shared memory holds (at least cols)
  int warps, team;  // of a CTA, of a team
  int phase_units;  // units of a phase; all of them: one phase
  int phase_rounds; // items a team walks per phase (several phases)
  int xs_offset, red_offset, acc_offset, ids_offset;  // shared memory
  int smem_bytes;
  uint64_t wait_limit_ns;
  int *status;
  int set_ctas;  // one matrix: CTAs of a column set
};

constexpr int kW4MaxSets = 32;   // column sets staged at a time
constexpr int kW4MaxXCols = 64;  // columns staged at a time

// Units of a warp's ring: 64 KB in flight an SM behind those in use.
__host__ __device__ constexpr int w4_depth(int r, int nt, int group) {
  return r * w4_parts(r, nt, group) == 1 ? 5 : 3;
}
__host__ __device__ constexpr int w4_row_bytes(int group) {
  return group == 32 ? 112 : group == 64 ? 96 : 64;
}
// Scales and zero points of a row: behind its weights, or with groups of 128
// behind the part's.
__host__ __device__ constexpr int w4_part_bytes(int r, int group) {
  return 16 * r * (w4_row_bytes(group) + (group == 128 ? 8 : 0));
}
__host__ __device__ constexpr int w4_ring_bytes(int r, int nt, int group) {
  return w4_depth(r, nt, group) * w4_parts(r, nt, group) * w4_part_bytes(r, group);
}

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// The first `bytes` of the source, zeros behind them (some instructions more).
__device__ __forceinline__ void cp_async_16_of(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_4_of(uint32_t dst, const void *src, uint32_t bytes) {
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
  const __half2 sixteenth = as_half2(0x2C002C00u);  // 1/16
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

__device__ __forceinline__ float gated(float gate, float up) {
  return gate / (1.f + expf(-gate)) * up;
}

// Row of W behind local row lr of block b: with the gated activation the
// first 8 R are gate rows, the others the up rows of the same outputs.
// Beyond the end: the last row, whose result is not stored.
template <int R>
__device__ __forceinline__ int w4_row(const W4Args &a, int block, int lr) {
  if (a.act == AR_ACT_SILU_MUL) {
    const int half = lr >= 8 * R ? 1 : 0;
    return min(block * 8 * R + lr - half * 8 * R, a.width - 1) + half * a.width;
  }
  return min(block * 16 * R + lr, a.N - 1);
}

// This CTA's share of the items (at most 4096 sets x 65536 blocks): of one
// column set's, where the sets are known to the host (none then unpacks the x
// of two: 16 x 4096 x 4096 in 11.2 us against 15 us), else of all.
template <bool EXPERTS>
__device__ __forceinline__ void w4_range(const W4Args &a, int nsets, int *first, int *end) {
  unsigned total = nsets * a.row_blocks, i = blockIdx.x, n = gridDim.x, before = 0;
  if constexpr (!EXPERTS) {
    n = a.set_ctas;
    before = i / n * a.row_blocks;
    i %= n;
    total = a.row_blocks;
  }
  const unsigned each = total / n;
  const unsigned more = total - each * n;
  *first = static_cast<int>(before + i * each + min(i, more));
  *end = *first + static_cast<int>(each + (i < more ? 1u : 0u));
}

// One output, by one warp: x as it is, eight products at a time in fp32, times
// their scale.
template <int ST, bool ZEROS>
__device__ float w4_dot(const W4Args &a, const uint4 *x, int64_t row) {
  const int shift = __ffs(a.K / a.ng / 8) - 1;  // eights of a group: 4, 8 or 16
  const uint32_t *q = reinterpret_cast<const uint32_t *>(a.q + row * (a.K / 2));
  float sum = 0.f;
#pragma unroll 4
  for (int k8 = threadIdx.x & 31; k8 < a.K / 8; k8 += 32) {
    const int64_t el = row * a.ng + (k8 >> shift);
    const float s =
        ST == AR_TYPE_F32
            ? __ldg(reinterpret_cast<const float *>(a.scales) + el)
            : __uint_as_float(uint32_t{__ldg(reinterpret_cast<const uint16_t *>(a.scales) + el)} << 16);
    const float z = ZEROS ? static_cast<float>(__ldg(a.zeros + el) & 15) : 8.f;
    const uint32_t word = __ldg(q + k8);
    float v[8], d = 0.f;
    unpack8(__ldg(x + k8), v);
#pragma unroll
    for (int j = 0; j < 8; ++j) d = fmaf(static_cast<float>(word >> 4 * j & 15u) - z, v[j], d);
    sum = fmaf(s, d, sum);
  }
  return warp_sum(sum);
}

// This CTA's outputs that are no finite numbers, again.  A scale of 2^95 or
// more times a sum of x as fp16 can pass fp32's end where the column's power
// of two would have brought the result back.  (bf16 and fp32 scales; 2^16 is
// fp16's largest.)  Behind the items, where it takes none of their registers
// (0 to 1.8 % of a call): the power of two of each product in front of its
// scale cost 0 to 8 % of every call, a second look at each item's sums 4 %.
template <int R, int ST, bool ZEROS, bool EXPERTS>
__device__ __noinline__ void w4_again(const W4Args &a, const int *sets, const int16_t *ids16) {
  const int lane = threadIdx.x & 31;
  const int outs = a.act == AR_ACT_SILU_MUL ? 8 * R : 16 * R;
  int item0, item1, e = 0;
  w4_range<EXPERTS>(a, EXPERTS ? sets[a.E] : 0, &item0, &item1);
  for (int item = item0 + (threadIdx.x >> 5); item < item1; item += blockDim.x >> 5) {
    const int set = item / a.row_blocks, block = item - set * a.row_blocks;
    if constexpr (EXPERTS)
      while (sets[e + 1] <= set) ++e;
    int col = -(EXPERTS ? set - sets[e] : set) * a.cols;  // of the next pair of the expert
    for (int p0 = 0; p0 < a.pairs && col < a.cols; p0 += 32) {
      uint32_t who = __ballot_sync(
          0xFFFFFFFFu, p0 + lane < a.pairs && (!EXPERTS || ids16[p0 + lane] == e));
      for (; who != 0 && col < a.cols; who &= who - 1, ++col) {
        if (col < 0) continue;
        const int pair = p0 + __ffs(who) - 1;
        const uint4 *x = a.x + static_cast<int64_t>(pair / a.k) * (a.K / 8);
        __nv_bfloat16 *to = a.out + static_cast<int64_t>(pair) * a.width + block * outs;
        const bool past = lane < outs && block * outs + lane < a.width &&
                          !(fabsf(__bfloat162float(to[lane])) < INFINITY);
        for (uint32_t odd = __ballot_sync(0xFFFFFFFFu, past); odd != 0; odd &= odd - 1) {
          const int o = __ffs(odd) - 1;
          const int64_t row = static_cast<int64_t>(e) * a.N + block * outs + o;
          float v = w4_dot<ST, ZEROS>(a, x, row);
          if (a.act == AR_ACT_SILU_MUL) v = gated(v, w4_dot<ST, ZEROS>(a, x, row + a.width));
          // x next to its largest may give inf - inf here alone.
          if (v == v && lane == 0) to[o] = __float2bfloat16_rn(v);
        }
      }
    }
  }
}

// A warp's way through its CTA's items [item0, item1): chunk by chunk, in
// each chunk phase by phase, in each phase the team's items, and of all their
// units in a row every team'th.  One phase: one chunk.
struct W4Walk {
  int item1, teams, team_warps, team, member;
  int base, end;   // the chunk
  int u0, u1;      // the phase's units
  int item, unit;  // where the warp is
  bool more;

  __device__ __forceinline__ int chunk_end(const W4Args &a, int first) const {
    if (a.phase_units >= a.units) return item1;
    const int set_end = (first / a.row_blocks + 1) * a.row_blocks;
    return min(item1, min(set_end, first + a.phase_rounds * teams));
  }
  __device__ __forceinline__ void start(const W4Args &a, int item0, int item1_, int warp) {
    item1 = item1_;
    team_warps = a.team;
    teams = a.warps / a.team;
    team = warp / a.team;
    member = warp % a.team;
    base = item0;
    end = chunk_end(a, item0);
    u0 = 0;
    u1 = a.phase_units;
    item = base + team;
    unit = member;
    more = item0 < item1;
    if (more) settle(a);
  }
  // From (item, unit) on, the first unit that exists.
  __device__ __forceinline__ void settle(const W4Args &a) {
    for (;;) {
      if (item >= end) {  // next phase, or next chunk
        u0 = u1;
        if (u0 >= a.units) {
          u0 = 0;
          base = end;
          more = base < item1;
          if (!more) return;
          end = chunk_end(a, base);
        }
        u1 = min(a.units, u0 + a.phase_units);
        item = base + team;
        unit = u0 + member;
      } else if (unit >= u1) {  // the team's warps take up the next item where this one left them
        unit -= u1 - u0;
        item += teams;
      } else {
        return;
      }
    }
  }
};

// ST: AR_TYPE_* of the scales; ZEROS: whether there are zero points.
template <int R, int NT, int G, int ST, bool ZEROS, bool EXPERTS>
__global__ void __launch_bounds__(kW4MaxWarps * 32, 1) k_w4_matvec(const __grid_constant__ W4Args a) {
  extern __shared__ __align__(16) unsigned char w4_smem[];
  constexpr int kDepth = w4_depth(R, NT, G), kParts = w4_parts(R, NT, G);
  constexpr int kPart = w4_part_bytes(R, G), kSlot = kParts * kPart;
  static_assert(kDepth * kSlot == w4_ring_bytes(R, NT, G), "the ring that the plan laid out");
  constexpr int kRowBytes = w4_row_bytes(G);
  constexpr int kGroups = kW4PartK / G;  // groups of a part
  constexpr int kRows = 16 * R;
  // Of local row lr: its scale words at lr * kScaleStride + kScaleAt, its
  // zero points kZeroAt behind them.
  constexpr int kScaleAt = G == 128 ? kRows * 64 : 64;
  constexpr int kScaleStride = G == 128 ? 8 : kRowBytes;
  constexpr int kZeroAt = G == 128 ? 4 : G == 64 ? 8 : 32;
  constexpr int kScaleBytes = ST == AR_TYPE_F32 ? 4 : 2;
  // Aligned words that hold a part's scales, or zero points, of one row.
  constexpr int kScaleWords = ST == AR_TYPE_F32 ? kGroups : kGroups == 1 ? 1 : kGroups / 2 + 1;
  constexpr int kZeroWords = kGroups == 1 ? 1 : 2;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int warps = a.warps, threads = warps * 32;
  const int teams = warps / a.team, team = warp / a.team, member = warp % a.team;

  const uint32_t ring = smem_addr(w4_smem) + warp * (kDepth * kSlot);
  uint4 *xs = reinterpret_cast<uint4 *>(w4_smem + a.xs_offset);
  // red[team][item & 1][member][column][row], sums[round of the phase][team][column][row]
  float *red = reinterpret_cast<float *>(w4_smem + a.red_offset);
  float *sums = reinterpret_cast<float *>(w4_smem + a.acc_offset);
  const int tile = a.cols * kRows;  // sums of an item

  // Experts: ids16[p] the expert of pair p (-1: none), sets[e] the number of
  // column sets before expert e, counts[e] its pairs.
  int16_t *ids16 = reinterpret_cast<int16_t *>(w4_smem + a.ids_offset);
  __shared__ int sets[EXPERTS ? AR_MAX_EXPERTS + 1 : 1];
  __shared__ int16_t counts[EXPERTS ? AR_MAX_EXPERTS : 1];
  // The staged sets: expert, first column, columns.
  __shared__ int set_expert[kW4MaxSets], set_col[kW4MaxSets + 1];
  __shared__ int set_count;
  __shared__ int col_pair[kW4MaxXCols];
  __shared__ int col_top[kW4MaxXCols];  // bits of a column's largest finite |x|
  __shared__ uint4 nothing[20];         // a unit of no column: zeros
  // Of team and buffer: all warps have left their sums, all have read them.
  __shared__ uint64_t full[kW4MaxWarps], empty[kW4MaxWarps];
  __shared__ int aborted;
  __shared__ bool col_odd[kW4MaxXCols];  // whether a column has an infinity or a NaN
  __shared__ bool again;                 // some output of another is no finite number

  int nsets = (a.pairs + a.cols - 1) / a.cols;
  if constexpr (!EXPERTS) {
    // The first units' lines on their way to L2 while the previous grid
    // drains: nothing enters this SM before the wait.
    int item, end;
    w4_range<EXPERTS>(a, nsets, &item, &end);
    item += team;
    if (item < end && (t & 1) == 0) {
      const int block = item % a.row_blocks;
      const int64_t row_bytes = a.K / 2;
      for (int d = 0, u = member; d < kDepth - 1 && u < a.phase_units; ++d, u += a.team) {
        const int64_t piece = static_cast<int64_t>(u) * (64 * kParts) + t * (16 * kParts);
#pragma unroll
        for (int i = 0; i < 2 * R; ++i)
          if (piece < row_bytes)
            prefetch_line(a.q + w4_row<R>(a, block, g + 8 * i) * row_bytes + piece);
      }
    }
  }
  if (tid < kW4MaxWarps) {
    mbar_init(&full[tid], a.team);
    mbar_init(&empty[tid], a.team);
  }
  if (tid < 20) nothing[tid] = make_uint4(0, 0, 0, 0);
  if (tid == 0) aborted = 0, again = false;
  if constexpr (EXPERTS) {
    for (int e = tid; e <= AR_MAX_EXPERTS; e += threads) sets[e] = 0;
    __syncthreads();
  }
  pdl_wait_prior_grid();
  pdl_launch_dependents();

  if constexpr (EXPERTS) {
    const int each = (a.E + 31) / 32;  // experts a lane counts up
    for (int p = tid; p < a.pairs; p += threads) {
      const int e = static_cast<int>(static_cast<uint32_t>(__ldg(a.ids + p)) -
                                     static_cast<uint32_t>(a.first));
      const bool ok = static_cast<uint32_t>(e) < static_cast<uint32_t>(a.E);
      ids16[p] = static_cast<int16_t>(ok ? e : -1);
      if (ok) atomicAdd(&sets[e], 1);
    }
    __syncthreads();
    if (warp == 0) {  // counts -> column sets before each expert
      int mine = 0;
      for (int i = 0; i < each; ++i) mine += (sets[lane * each + i] + a.cols - 1) / a.cols;
      int before = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, before, o);
        if (lane >= o) before += v;
      }
      const int all = __shfl_sync(0xFFFFFFFFu, before, 31);
      before -= mine;
      __syncwarp();
      for (int i = 0; i < each; ++i) {
        const int e = lane * each + i;
        if (e < a.E) {
          const int n = sets[e];
          counts[e] = static_cast<int16_t>(n);
          sets[e] = before;
          before += (n + a.cols - 1) / a.cols;
        }
      }
      __syncwarp();
      if (lane == 0) sets[a.E] = all;
    }
    __syncthreads();
    nsets = sets[a.E];
    // Pairs without an expert here: zero rows, spread over the grid.
    for (int p = blockIdx.x; p < a.pairs; p += gridDim.x)
      if (ids16[p] < 0)
        for (int n = tid; n < a.width; n += threads)
          a.out[static_cast<int64_t>(p) * a.width + n] = __float2bfloat16_rn(0.f);
  } else {
    __syncthreads();  // the barriers are there
  }
  int item0, item1;
  w4_range<EXPERTS>(a, nsets, &item0, &item1);
  // Checking build: the launch has the plan's warps, whole teams, room for a
  // column set, and the regions of shared memory that the kernel walks, one
  // behind the other.
  uint32_t dynamic_bytes;
  asm volatile("mov.u32 %0, %%dynamic_smem_size;" : "=r"(dynamic_bytes));
  const int tile_bytes = tile * static_cast<int>(sizeof(float));
  if (!in_bounds(
          threads == static_cast<int>(blockDim.x) && warps <= kW4MaxWarps && warps % a.team == 0 &&
              a.cols <= 8 * NT && a.cols <= a.x_cols && a.x_cols <= kW4MaxXCols &&
              warps * kDepth * kSlot <= a.xs_offset &&
              a.xs_offset + a.x_cols * min(a.phase_units, a.units) * kParts * 256 <= a.red_offset &&
              a.red_offset + (a.team > 1 ? 2 * warps * tile_bytes : 0) <= a.acc_offset &&
              a.acc_offset + (a.phase_units < a.units ? a.phase_rounds * teams * tile_bytes : 0) <=
                  a.ids_offset &&
              a.ids_offset + (EXPERTS ? 2 * a.pairs : 0) <= a.smem_bytes &&
              static_cast<uint32_t>(a.smem_bytes) <= dynamic_bytes &&
              (!EXPERTS || (nsets >= 0 && nsets <= a.E + a.pairs / a.cols)),
          a.status))
    item1 = item0;
  // Checking build: a row of out.
  auto pair_of = [&](int col) -> int {
    const int p = col_pair[col];
    return in_bounds(p >= 0 && p < a.pairs, a.status) ? p : 0;
  };

  // The expert of a column set.
  auto expert_of = [&](int set) -> int {
    if constexpr (!EXPERTS) return 0;
    int lo = 0, hi = a.E;  // sets[lo] <= set < sets[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sets[mid] <= set) lo = mid;
      else hi = mid;
    }
    return lo;
  };

  const bool act = a.act == AR_ACT_SILU_MUL;
  const int outs = act ? 8 * R : kRows;  // outputs of an item's column

  // The fetching side of the ring, `to_come` units of an item at a time.
  W4Walk walk;
  walk.start(a, item0, item1, warp);
  const int64_t row_bytes = a.K / 2;
  int to_come = 0, f_unit = 0;
  int f_set = -1;
  int64_t f_first = 0;           // first row of W of the set's expert
  const uint8_t *f_q = nullptr;  // this lane's 16 bytes of the unit in the expert's first row
  uint32_t f_off[2 * R];         // the rows' distances, in 16 bytes
  // The unit's scales and zero points of one row of a part: part lane / 16
  // (one row tile) or row `lane`.
  const int s_part = kParts > 1 ? lane / kRows : 0;
  const uint8_t *f_s = nullptr, *f_z = nullptr;
  bool f_plain = false;          // neither ends inside a unit nor near the end of its arrays
  uint32_t f_slot = ring;
  // Points at the rows of the walk's item and takes its units.
  auto next_item = [&]() {
    const int set = walk.item / a.row_blocks, block = walk.item - set * a.row_blocks;
    if (set != f_set) {
      f_set = set;
      f_first = static_cast<int64_t>(expert_of(set)) * a.N;
    }
    f_unit = walk.unit;
    to_come = (walk.u1 - walk.unit + a.team - 1) / a.team;
    f_q = a.q + f_first * row_bytes + t * 16 + f_unit * (64 * kParts);
#pragma unroll
    for (int i = 0; i < 2 * R; ++i)
      f_off[i] = static_cast<uint32_t>(w4_row<R>(a, block, g + 8 * i)) *
                 static_cast<uint32_t>(row_bytes >> 4);
    const int64_t el = (f_first + w4_row<R>(a, block, lane & (kRows - 1))) * a.ng +
                       (f_unit * kParts + s_part) * kGroups;
    f_s = a.scales + el * kScaleBytes;
    if constexpr (ZEROS) f_z = a.zeros + el;
    f_plain = __all_sync(0xFFFFFFFFu, el + a.ng + 16 <= a.scale_count) && a.K % (kParts * kW4PartK) == 0;
    walk.unit += to_come * a.team;
    walk.settle(a);
  };
  auto word_of = [](const uint8_t *p) -> const uint8_t * {
    return reinterpret_cast<const uint8_t *>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t{3});
  };
  auto fetch = [&]() {
    if (to_come == 0 && walk.more) next_item();
    if (to_come > 0) {
      --to_come;
      const uint32_t to = f_slot + g * kRowBytes + t * 16;
      const uint32_t to_s = f_slot + s_part * kPart + kScaleAt + (lane & (kRows - 1)) * kScaleStride;
      const uint8_t *ws = word_of(f_s), *wz = word_of(f_z);
      if (f_plain) {
#pragma unroll
        for (int i = 0; i < 2 * R; ++i)
#pragma unroll
          for (int j = 0; j < kParts; ++j)
            cp_async_16(to + j * kPart + 8 * i * kRowBytes,
                        f_q + static_cast<uint64_t>(f_off[i]) * 16 + j * 64);
        if (kParts * kRows == 32 || lane < kRows) {
#pragma unroll
          for (int i = 0; i < kScaleWords; ++i) cp_async_4(to_s + 4 * i, ws + 4 * i);
          if constexpr (ZEROS) {
#pragma unroll
            for (int i = 0; i < kZeroWords; ++i) cp_async_4(to_s + kZeroAt + 4 * i, wz + 4 * i);
          }
        }
      } else {
        // Zeros behind the row's end; words cut off at the end of the arrays.
#pragma unroll
        for (int j = 0; j < kParts; ++j) {
          const bool here = (f_unit * kParts + j) * 64 + t * 16 < static_cast<int>(row_bytes);
#pragma unroll
          for (int i = 0; i < 2 * R; ++i)
            cp_async_16_of(to + j * kPart + 8 * i * kRowBytes,
                           here ? f_q + static_cast<uint64_t>(f_off[i]) * 16 + j * 64 : a.q,
                           here ? 16u : 0u);
        }
        auto words = [&](uint32_t dst, const uint8_t *w, const uint8_t *end, int n) {
          for (int i = 0; i < n; ++i) {
            const int64_t left = end - (w + 4 * i);
            if (left > 0)
              cp_async_4_of(dst + 4 * i, w + 4 * i, left < 4 ? static_cast<uint32_t>(left) : 4u);
          }
        };
        if (kParts * kRows == 32 || lane < kRows) {
          words(to_s, ws, a.scales + a.scale_count * kScaleBytes, kScaleWords);
          if constexpr (ZEROS) words(to_s + kZeroAt, wz, a.zeros + a.scale_count, kZeroWords);
        }
      }
      f_unit += a.team;
      f_q += a.team * (64 * kParts);
      f_s += a.team * (kParts * kGroups * kScaleBytes);
      if constexpr (ZEROS) f_z += a.team * (kParts * kGroups);
      f_slot += kSlot;
      if (f_slot == ring + kDepth * kSlot) f_slot = ring;
    }
    cp_async_commit();  // an empty group at the end keeps the count
  };
#pragma unroll 1
  for (int i = 0; i < kDepth - 1; ++i) fetch();

  // Units [u0, u1) of the first n columns into shared memory, as fp16 times
  // their powers of two: [part][column][step][lane], odd columns with the
  // steps of a pair exchanged (no bank conflicts between two columns).  A
  // column's eights go to one warp, or to as many as there are for it; eight
  // loads of a lane are under way at a time.
  auto stage = [&](int u0, int u1, int n) {
    const int pieces = (u1 - u0) * (16 * kParts);  // eights of a column
    const int before = u0 * (16 * kParts);
    const int share = n < warps ? warps / n : 1;  // warps of a column
    const int step = share * 32, j0 = warp % share * 32 + lane;
    auto place = [&](int j, int col) -> uint4 * {
      const int to = step_lane<G>(j & 15);
      return xs + ((j >> 4) * a.x_cols + col) * 16 + (to ^ ((col & 1) << 2));
    };
    for (int col = warp / share; col < n; col += warps / share) {
      const uint4 *row = a.x + static_cast<int64_t>(pair_of(col) / a.k) * (a.K / 8) + before;
      const int whole = min(pieces, a.K / 8 - before);  // eights that the row has here
      uint32_t tops = 0;  // the largest magnitudes of the even and of the odd elements
      for (int j = j0; j < pieces; j += 8 * step) {
        uint4 w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int at = j + i * step;
          w[i] = make_uint4(0, 0, 0, 0);
          if (at < whole) w[i] = __ldg(row + at);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int at = j + i * step;
          if (at >= pieces) break;
          const uint4 v = w[i];
          tops = __vmaxu2(tops, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                         __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
          *place(at, col) = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                                       __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
        }
      }
      uint32_t top = max(tops & 0xFFFFu, tops >> 16);
      if (top >= 0x7F80u) {  // an infinity or a NaN: the largest of the others
        top = 0, col_odd[col] = true;
        for (int j = j0; j < whole; j += step) {
          const uint4 v = __ldg(row + j);
          const uint32_t e[4] = {v.x, v.y, v.z, v.w};
          for (int i = 0; i < 8; ++i) {
            const uint32_t h = e[i / 2] >> (i % 2 * 16) & 0x7FFFu;
            if (h < 0x7F80u) top = max(top, h);
          }
        }
      }
      top = __reduce_max_sync(0xFFFFFFFFu, top) << 16;  // a bf16 is the top half of an fp32
      if (lane == 0) {
        if (share == 1) col_top[col] = static_cast<int>(top);
        else atomicMax(&col_top[col], static_cast<int>(top));
      }
    }
    if (share > 1) __syncthreads();
    else __syncwarp();
    for (int col = warp / share; col < n; col += warps / share) {
      const float down = __int_as_float((127 - exponent_of(col_top[col])) << 23);
#pragma unroll 4
      for (int j = j0; j < pieces; j += step) {  // what this lane has put there
        uint4 *to = place(j, col);
        uint4 v = *to;
        v.x = halves_of(v.x, down), v.y = halves_of(v.y, down);
        v.z = halves_of(v.z, down), v.w = halves_of(v.w, down);
        *to = v;
      }
    }
    __syncthreads();
  };

  // fp16 scales cannot pass fp32's end.
  auto put = [&](__nv_bfloat16 *to, float v, int col) {
    *to = __float2bfloat16_rn(v);
    if constexpr (ST != AR_TYPE_F16)
      if (!(fabsf(v) < INFINITY) && !col_odd[col]) again = true;
  };

  int done = 0;  // items of this team that its warps have left (its buffers' phases)
  struct Item {
    int block, col, ncols, round;
  };
  // This warp's part of adding up item `it`, the team's number `n`, once
  // every warp has left its sums.
  auto gather = [&](const Item &it, int n, bool first, bool last) {
    const int at = team * 2 + (n & 1);
    mbar_wait_bounded(&full[at], (n >> 1) & 1, &aborted, a.wait_limit_ns, a.status);
    const float *buf = red + at * a.team * tile;
    float *sum = sums + (it.round * teams + team) * tile;
    auto sum_of = [&](int col, int row) -> float {
      const float *p = buf + col * kRows + row;
      float v = p[0];
      for (int w = 1; w < a.team; ++w) v += p[w * tile];
      if (!first) v += sum[col * kRows + row];
      if (!last) sum[col * kRows + row] = v;
      return v;
    };
    for (int i = member * 32 + lane; i < it.ncols * outs; i += a.team * 32) {
      const int col = i / outs, o = i - col * outs;
      float v = sum_of(col, o);
      if (act) {
        const float up = sum_of(col, o + 8 * R);
        if (last) v = gated(v, up);
      }
      const int n0 = it.block * outs + o;
      if (last && n0 < a.width)
        put(a.out + static_cast<int64_t>(pair_of(it.col + col)) * a.width + n0, v, it.col + col);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[at]);
  };

  uint32_t slot = ring;
#pragma unroll 1
  for (int base = item0; base < item1;) {
    const int chunk = walk.chunk_end(a, base);  // depends on base alone
    for (int u0 = 0; u0 < a.units; u0 += a.phase_units) {
      const int u1 = min(a.units, u0 + a.phase_units), nunits = u1 - u0;
      const bool first = u0 == 0, last = u1 == a.units;
      int c_unit = member;           // of the phase
      int item = base + team, round = 0;
      Item left = {0, 0, 0, 0};      // the team's item before, not added up yet
      bool pending = false;
#pragma unroll 1
      for (int at = base; at < chunk;) {
        // The column sets from item `at` on that fit together: [at, end).
        const int set0 = at / a.row_blocks;
        if (at != item0 || u0 != 0) __syncthreads();  // nobody uses the sets before any more
        if (warp == 0) {
          const int set = set0 + lane;
          const bool there = set < nsets && set * a.row_blocks < chunk;
          int n = 0;
          if (there) {
            const int e = expert_of(set);
            if constexpr (EXPERTS) n = min(a.cols, counts[e] - (set - sets[e]) * a.cols);
            else n = min(a.cols, a.pairs - set * a.cols);
            set_expert[lane] = e;
          }
          int before = n;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, before, o);
            if (lane >= o) before += v;
          }
          const uint32_t fit = __ballot_sync(0xFFFFFFFFu, there && before <= a.x_cols);
          if (lane == 0) {
            set_count = __popc(fit);
            set_col[0] = 0;
          }
          if (fit >> lane & 1u) set_col[lane + 1] = before;
        }
        for (int c = tid; c < kW4MaxXCols; c += threads) {
          col_top[c] = 0;
          if (u0 == 0) col_odd[c] = false;  // later phases: the same columns
          if constexpr (!EXPERTS) col_pair[c] = set0 * a.cols + c;  // the sets are full but the last
        }
        __syncthreads();
        const int count = set_count;
        const int end = min(chunk, (set0 + count) * a.row_blocks);
        if constexpr (EXPERTS) {
          for (int i = warp; i < count; i += warps) {  // the sets' pairs, in order
            const int c0 = set_col[i], n = set_col[i + 1] - c0;
            const int e = set_expert[i], skip = (set0 + i - sets[e]) * a.cols;
            int seen = 0;
            for (int p0 = 0; p0 < a.pairs && seen < skip + n; p0 += 32) {
              const bool is = p0 + lane < a.pairs && ids16[p0 + lane] == e;
              const uint32_t who = __ballot_sync(0xFFFFFFFFu, is);
              const int k = seen + __popc(who & ((1u << lane) - 1u)) - skip;
              if (is && k >= 0 && k < n) col_pair[c0 + k] = p0 + lane;
              seen += __popc(who);
            }
          }
          __syncthreads();
        }
        // Checking build: the staged sets and their columns have room, and the
        // rounds of a phase sums of their own.
        if (!in_bounds(count >= 1 && count <= kW4MaxSets && set_col[count] <= a.x_cols &&
                           (u1 - u0) <= a.phase_units &&
                           (a.phase_units >= a.units ||
                            (end - base + teams - 1) / teams <= a.phase_rounds),
                       a.status))
          break;  // the same in every thread
        stage(u0, u1, set_col[count]);

#pragma unroll 1
        for (; item < end; item += teams, ++round) {
          const int set = item / a.row_blocks, si = set - set0;
          const Item it = {item - set * a.row_blocks, set_col[si], set_col[si + 1] - set_col[si], round};
          // This lane's eights of x: column g of each tile, or zeros; even
          // and odd steps.
          uint32_t xe[NT], xo[NT], xstep[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const int col = it.col + n * 8 + g;
            const bool in = n * 8 + g < it.ncols;
            const uint32_t p = in ? smem_addr(xs + col * 16 + t) : smem_addr(nothing + 4);
            const int odd = in ? (col & 1) * 64 : 0;
            xe[n] = p + odd;
            xo[n] = p - odd;
            xstep[n] = in ? a.x_cols * 256 : 0;
          }
          // Low bits of the rows' first group numbers.
          const int first_row = set_expert[si] * a.N;
          int el_low[R][2];
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              el_low[r][h] =
                  ((first_row + w4_row<R>(a, it.block, r * 16 + h * 8 + g)) & 3) * (a.ng & 3);
          float acc[R][NT][4];
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int c = 0; c < 4; ++c) acc[r][n][c] = 0.f;
#pragma unroll 1
          for (; c_unit < nunits; c_unit += a.team) {
            cp_async_wait<kDepth - 2>();
            __syncwarp();  // every lane's copies are here, and the slot before is free
            fetch();
#pragma unroll
            for (int j = 0; j < kParts; ++j) {
              const uint32_t part = slot + j * kPart;
              uint4 b[4][NT];
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                const uint32_t off = (c_unit * kParts + j) * xstep[n];
                b[0][n] = lds_128(xe[n] + off);
                b[1][n] = lds_128(xo[n] + off + 64);
                b[2][n] = lds_128(xe[n] + off + 128);
                b[3][n] = lds_128(xo[n] + off + 192);
              }
              const int group0 = ((u0 + c_unit) * kParts + j) * kGroups;
#pragma unroll
              for (int r = 0; r < R; ++r) {
                uint32_t w0[4], w1[4];
                load_words<G>(w0, part + (r * 16 + g) * kRowBytes, t);
                load_words<G>(w1, part + (r * 16 + 8 + g) * kRowBytes, t);
                const uint32_t sc = part + kScaleAt + (r * 16 + g) * kScaleStride;
#pragma unroll
                for (int gi = 0; gi < kGroups; ++gi) {
                  // Scale and zero point of the two rows' group.
                  float s[2];
                  Offsets o[2];
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    const uint32_t p = sc + h * 8 * kScaleStride;
                    const int low = el_low[r][h] + group0;
                    if constexpr (ST == AR_TYPE_F32) {
                      s[h] = __uint_as_float(lds_32(p + gi * 4));
                    } else if constexpr (G == 128) {
                      // The upper or the lower half of the word, as the upper one.
                      const uint32_t v = __byte_perm(lds_32(p), 0, (low & 1) * 0x2200 + 0x1044);
                      s[h] = ST == AR_TYPE_BF16
                                 ? __uint_as_float(v)
                                 : __half2float(__ushort_as_half(static_cast<unsigned short>(v >> 16)));
                    } else {
                      const uint32_t v = lds_16(p + (el_low[r][h] & 1) * 2 + gi * 2);
                      s[h] = ST == AR_TYPE_BF16
                                 ? __uint_as_float(v << 16)
                                 : __half2float(__ushort_as_half(static_cast<unsigned short>(v)));
                    }
                    // Behind the row's end stands another row's scale.
                    if (kParts * kGroups > 1 && group0 + gi >= a.ng) s[h] = 0.f;
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
                      if (i == gi * kSteps)
                        mma_first(d[n], p[0], q[0], p[1], q[1], b[i][n].x, b[i][n].y);
                      else
                        mma_next(d[n], p[0], q[0], p[1], q[1], b[i][n].x, b[i][n].y);
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
            slot += kSlot;
            if (slot == ring + kDepth * kSlot) slot = ring;
          }
          c_unit -= nunits;
          // Back to the columns' powers of two.
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int col = min(it.col + n * 8 + 2 * t + c, kW4MaxXCols - 1);
              const float up = __int_as_float((127 + exponent_of(col_top[col])) << 23);
#pragma unroll
              for (int r = 0; r < R; ++r) acc[r][n][c] *= up, acc[r][n][c + 2] *= up;
            }

          if (a.team == 1) {  // the warp has the whole sums of the phase
            float *sum = sums + (round * teams + team) * tile;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const int col = n * 8 + 2 * t + c;
                if (col >= it.ncols) continue;
                const int o0 = it.block * outs + g;
                __nv_bfloat16 *to = a.out + static_cast<int64_t>(pair_of(it.col + col)) * a.width + o0;
                float v[R][2];
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    float *p = sum + col * kRows + r * 16 + h * 8 + g;
                    v[r][h] = acc[r][n][c + 2 * h];
                    if (!first) v[r][h] += *p;
                    if (!last) *p = v[r][h];
                  }
                if (!last) continue;
                if (act) {  // R = 1: gate and up rows eight apart, R = 2: sixteen
                  if constexpr (R == 1) {
                    if (o0 < a.width) put(to, gated(v[0][0], v[0][1]), it.col + col);
                  } else {
                    if (o0 < a.width) put(to, gated(v[0][0], v[1][0]), it.col + col);
                    if (o0 + 8 < a.width) put(to + 8, gated(v[0][1], v[1][1]), it.col + col);
                  }
                } else {
#pragma unroll
                  for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                      if (o0 + r * 16 + h * 8 < a.width)
                        put(to + r * 16 + h * 8, v[r][h], it.col + col);
                }
              }
            continue;
          }
          // The sums go to the team's buffer, which every warp has read since
          // the item before last; then the item before is added up.
          const int at2 = team * 2 + (done & 1);
          if (done >= 2)
            mbar_wait_bounded(&empty[at2], ((done >> 1) + 1) & 1, &aborted, a.wait_limit_ns, a.status);
          float *buf = red + (at2 * a.team + member) * tile;
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const int col = n * 8 + 2 * t + (c & 1), row = r * 16 + (c >> 1) * 8 + g;
                if (col < it.ncols) buf[col * kRows + row] = acc[r][n][c];
              }
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[at2]);
          if (pending) gather(left, done - 1, first, last);
          left = it;
          pending = true;
          ++done;
        }
        if (pending) {  // col_pair is about to change
          gather(left, done - 1, first, last);
          pending = false;
        }
        at = end;
      }
    }
    base = chunk;
  }
  cp_async_wait<0>();
  if constexpr (ST != AR_TYPE_F16) {
    __syncthreads();
    if (again) w4_again<R, ST, ZEROS, EXPERTS>(a, sets, ids16);
  }
}

using W4Kernel = void (*)(W4Args);
// Row tiles 1 or 2 (1 with groups of 32, whose scales would fill the
// registers), column tiles 1 or 2.
template <int ST, bool ZEROS, bool EXPERTS>
inline W4Kernel w4_pick(int r, int nt, int group) {
  if (group == 32)
    return nt == 1 ? &k_w4_matvec<1, 1, 32, ST, ZEROS, EXPERTS>
                   : &k_w4_matvec<1, 2, 32, ST, ZEROS, EXPERTS>;
  if (group == 64)
    return nt == 1 ? (r == 1 ? &k_w4_matvec<1, 1, 64, ST, ZEROS, EXPERTS>
                             : &k_w4_matvec<2, 1, 64, ST, ZEROS, EXPERTS>)
                   : (r == 1 ? &k_w4_matvec<1, 2, 64, ST, ZEROS, EXPERTS>
                             : &k_w4_matvec<2, 2, 64, ST, ZEROS, EXPERTS>);
  return nt == 1 ? (r == 1 ? &k_w4_matvec<1, 1, 128, ST, ZEROS, EXPERTS>
                           : &k_w4_matvec<2, 1, 128, ST, ZEROS, EXPERTS>)
                 : (r == 1 ? &k_w4_matvec<1, 2, 128, ST, ZEROS, EXPERTS>
                           : &k_w4_matvec<2, 2, 128, ST, ZEROS, EXPERTS>);
}

}  // namespace arn
