// Products of 8-bit integers on the tensor cores (ar_i8_matmul above a few
// tokens): the kernel.
//
// The part's own 8-bit integer rate is far below its 16-bit floating-point
// rate, so the bytes are multiplied as fp16: every byte is exact there, a
// product of two has 14 bits, and fp32 adds whole numbers exactly up to 2^24.
//
// Beyond 2^24 the accumulator drops what is below its step, 16 products at a time
// (16384 k of random bytes of 64 to 127: 464 off 1.5e8).  It is left so.  Sums that
// are exact for any data were built and measured: taken into other sums every 1024 k
// below 256 tokens, and with 256, whose accumulator leaves no tensor memory for that,
// where a bound from the operands' squares asks for it.  One CTA a tile took 4 to
// 15 % longer, pairs of 64 and 128 tokens 9 to 46 %, of 256 tokens 2 to 4 %, at
// 16384 k 2 to 46 %; sums of a layer's data stay some thirty times below 2^24.
//
// The tile.  The weights' rows are the 128 rows of the accumulator (256 of a
// pair of CTAs, each holding its own 128), the tokens its columns.  So one
// kernel serves from 16 tokens, where the weights' bytes are the bound and
// each is read once, to prompts, where the tensor cores are.  A pair shares the
// tokens' operand, each CTA unpacking half of it: above 32 tokens a CTA by itself
// spends its time moving that operand through shared memory (128 x 7168 x 7168:
// 23.8 us, pairs 17.3 us).
//
// The operands are unpacked on the way.  TMA brings boxes of 64 rows x 128
// bytes of w and as many rows of x as the CTA has tokens (128-byte swizzle; what
// lies behind the arrays' ends comes as zeros, which add nothing).  Four warps
// turn a stage of w into fp16 in tensor memory, from where the tensor core takes
// its A operand: a thread is a row, as in tensor memory, so unpacked weights,
// twice the bytes, never pass through shared memory.  They also turn x into the
// swizzled fp16 tile of the B operand.  A byte b becomes 1024 + (b + 128) by a
// byte permutation under the exponent of 1024, and one half2 subtraction leaves
// b (a published method: Kim, Henry, Fahim and Awadalla, "Who Says Elephants
// Can't Run", 2022).
//
// Roles: a warp issues the loads, a warp the products, teams of four warps unpack
// a stage each in turn, and of a pair four more warps write the outputs while the
// next tile's operands are unpacked, gated with the teams' help.  Between them
// rings of mbarriers, every wait bounded.  A pair of CTAs is persistent and takes
// tiles in turn; one CTA takes one tile.  With few tiles a cluster of `split` CTAs
// or pairs takes one, each a part of K, and they add the parts up through the
// cluster's shared memory, in a fixed order.
//
// Measured: 8192 x 6144 x 8192 in 422 us, 1955 TFLOP/s (a library's bf16 product
// of that rate: 1933); a stage of 128 k of a full pair takes 1030 clocks, 1024 of
// them the tensor core's, and shared memory is in use for as many: 32 KB in, out,
// unpacked and read again; gated, 8192 x 6144 x 16384, 823 us, 2003 TFLOP/s.
// 16 x 6144 x 32768 gated in 35.3 us, 5.7 TB/s: memory, and 5 us from the launch to
// the first bytes and from the last ones to the outputs.
#pragma once

#include <cuda.h>

#include "i8_matmul.cuh"

namespace arn {

struct I8TensorArgs {
  CUtensorMap w_map, x_map;
  I8Args a;
  int tiles_n, tiles_m;  // tiles of channels, of tokens
  int split;             // parts of K, a cluster's CTAs or pairs (1: none)
  int group;             // token tiles that are walked together (pairs)
  I8Waits waits;
};

constexpr int kI8TileRows = 128;  // channels of a CTA
constexpr int kI8StepK = 128;     // k of a stage
constexpr int kI8RawW = kI8TileRows * kI8StepK;
// Stages whose weights are prefetched before the previous grid's end (32 tokens,
// 32768 x 6144 gated: 35.7 us, 36.4 us without).
constexpr int kI8Prefetch = 3;

// NT: tokens of a tile; PAIR: two CTAs share it.
template <int NT, bool PAIR>
struct I8Shape {
  static constexpr int kTokens = PAIR ? NT / 2 : NT;  // tokens whose x this CTA holds
  // Teams of four warps that unpack, and the stages of the rings.  A team
  // always meets its own raw slots again: loads land in any order, and a wait
  // on a slot whose last but one load is still another team's to see would
  // take that load's phase for the one before it.  (Operand slots are given
  // back in order.)
  static constexpr int kTeams = PAIR ? 3 : 2;
  static constexpr int kOps = 3;
  static constexpr int kRaw = !PAIR ? 4 : NT <= 128 ? 6 : 3;
  static_assert(kRaw % kTeams == 0 && kTeams <= kOps && kTeams <= 3, "a team's slots");
  static_assert(kRaw <= 6 && kOps <= 3, "barriers");
  static constexpr int kOutWarp0 = 4 + 4 * kTeams;    // of a pair's warps that write
  static constexpr int kWarps = kOutWarp0 + (PAIR ? 4 : 0);
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kRawX = kTokens * kI8StepK;
  static constexpr int kRawBytes = kI8RawW + kRawX;
  static constexpr int kOpBytes = kTokens * kI8StepK * 2;
  static constexpr int kAccCols = NT < 32 ? 32 : NT;
  static constexpr int kOpCols = kI8StepK / 2;
  static constexpr int kCols = kAccCols + kOps * kOpCols <= 256 ? 256 : 512;
  static constexpr int kBuffer = (PAIR ? 32 : 16) * 128 * 4;    // one of i8_write's
  static constexpr int kExchange = PAIR ? 2 * kBuffer : 0;
  // One CTA a tile: the parts of a tile, in the rings' place.
  static constexpr int kRings = kRaw * kRawBytes + kOps * kOpBytes;
  static constexpr int kSmem = 1024 + kRings + kExchange;
  static constexpr int kCtasPerSm = kCols == 256 && kSmem <= 113 * 1024 ? 2 : 1;
  static_assert(PAIR || 2 * NT * kI8TileRows * 4 <= kRings, "the parts of a tile fit the rings");
  static_assert(kSmem + NT * 4 + 512 + 256 <= 227 * 1024, "shared memory of a CTA");
  static_assert(kAccCols + kOps * kOpCols <= 512, "tensor memory");
  // CTAs that fit an SM's shared memory together never ask for more tensor
  // memory than it has, whichever of these kernels they are of: an allocation
  // could otherwise wait for one that waits for it.
  static_assert(kCols == 256 ? kSmem > 76 * 1024 : kSmem > 152 * 1024, "tensor memory of an SM");
};

// --- PTX ------------------------------------------------------------------------

__device__ __forceinline__ bool i8_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

// mbar_wait_bounded for barriers that the cluster's CTAs and the tensor core
// arrive at, many times a tile: the clock, whose reading takes about as long
// as a stage, is looked at once in 64 tries.
__device__ __forceinline__ bool i8_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                        uint64_t limit_ns, int *status) {
  uint64_t t0 = 0;
  for (uint32_t tries = 1; !i8_try_wait(bar, parity); ++tries) {
    if (*abort_flag) return false;
    if (tries % 64 == 0) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > limit_ns) {
        *abort_flag = 1;
        if (status) atomicExch(status, AR_ERR_TIMEOUT);
        return false;
      }
    }
  }
  return true;
}

__device__ __forceinline__ uint32_t i8_mapa(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void i8_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// At another CTA's barrier.  It announces operands that this CTA's own tensor
// core reads, or reads that have ended, and so needs no release at the
// cluster's scope, which waits 1000 clocks and more for the thread's accesses
// to memory (it took 40 % of a pair's time).
__device__ __forceinline__ void i8_arrive_cluster(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

__device__ __forceinline__ void i8_load_box(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void i8_prefetch_box(const CUtensorMap *map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x),
               "r"(y)
               : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void i8_tmem_alloc(uint32_t slot, uint32_t cols) {
  if constexpr (PAIR) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
}
template <bool PAIR>
__device__ __forceinline__ void i8_tmem_free(uint32_t tmem, uint32_t cols) {
  if constexpr (PAIR)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
}

__device__ __forceinline__ void i8_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void i8_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// D += A B^T with A in tensor memory: 16 k.
template <bool PAIR>
__device__ __forceinline__ void i8_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
        : "memory");
}

// Arrives at `bar` (of both CTAs of a pair, `rank` and the next) once this
// thread's products so far are done.
template <bool PAIR>
__device__ __forceinline__ void i8_commit(uint32_t bar, uint32_t rank) {
  if constexpr (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(bar), "h"(static_cast<uint16_t>(3u << rank))
        : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}

// At a barrier of this CTA alone.
template <bool PAIR>
__device__ __forceinline__ void i8_commit_here(uint32_t bar) {
  if constexpr (PAIR)
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                 : "memory");
  else
    i8_commit<false>(bar, 0);
}

__device__ __forceinline__ void i8_tmem_store16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void i8_tmem_load32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void i8_tmem_load16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ uint4 i8_lds(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void i8_sts(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// One lane of a warp whose lanes are all here.  Tensor core and copy
// instructions issued under it take a few clocks each; under a plain test of
// the lane number they took 90.
__device__ __forceinline__ bool i8_elect() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// The cluster's barrier where nothing but the reads and copies that its threads
// have waited for is ordered by it: with a release an arrival waits for the
// thread's stores to memory, 2000 clocks.
__device__ __forceinline__ void i8_cluster_arrive() {
  __syncwarp();  // it takes whole warps
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void i8_cluster_wait() {
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// Four bytes as four fp16, in order.
__device__ __forceinline__ void i8_unpack(uint32_t v, uint32_t &lo, uint32_t &hi) {
  const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
  const uint32_t u = v ^ 0x80808080u;
  uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), off);
  const __half2 y = __hsub2(*reinterpret_cast<__half2 *>(&b), off);
  lo = *reinterpret_cast<const uint32_t *>(&x);
  hi = *reinterpret_cast<const uint32_t *>(&y);
}

// --- the kernel -----------------------------------------------------------------

struct I8Barriers {
  uint64_t raw_full[6], raw_empty[6], op_full[3], op_empty[3], acc_full, acc_empty, parts, quiet;
  uint32_t tmem;
  int abort;
};

template <typename OUT>
__device__ __forceinline__ OUT i8_out(float v);
template <>
__device__ __forceinline__ float i8_out<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 i8_out<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half i8_out<__half>(float v) {
  return __float2half_rn(v);
}

// A barrier of a team's four warps (its number in the instruction: a register
// would count as all sixteen).
__device__ __forceinline__ void i8_team_sync(int team) {
  if (team == 0)
    asm volatile("bar.sync 1, 128;" ::: "memory");
  else if (team == 1)
    asm volatile("bar.sync 2, 128;" ::: "memory");
  else if (team == 2)
    asm volatile("bar.sync 3, 128;" ::: "memory");
  else
    asm volatile("bar.sync 4, 128;" ::: "memory");
}
// Of all warps but the first four of a pair's CTA.
__device__ __forceinline__ void i8_teams_sync() { asm volatile("bar.sync 5, 512;" ::: "memory"); }

// Eight, or four fp32, outputs in a row.
template <typename OUT>
__device__ __forceinline__ uint4 i8_pack(const float *y);
template <>
__device__ __forceinline__ uint4 i8_pack<float>(const float *y) {
  return make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]),
                    __float_as_uint(y[3]));
}
template <>
__device__ __forceinline__ uint4 i8_pack<__nv_bfloat16>(const float *y) {
  const float f[8] = {y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7]};
  return pack16<__nv_bfloat16>(f);
}
template <>
__device__ __forceinline__ uint4 i8_pack<__half>(const float *y) {
  const float f[8] = {y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7]};
  return pack16<__half>(f);
}

// Rows that begin anywhere: `room` channels, at most kCh, of `left` tokens from
// `stage` to `to`, element by element; nothing at or behind `end`.
template <typename OUT, int kCh, int COLS>
__device__ __forceinline__ void i8_copy_out(OUT *to, const OUT *stage, int64_t width, int left, int64_t room,
                                            const OUT *end, int row, int *status) {
  const int c = row % kCh;
#pragma unroll 1
  for (int j0 = 0; j0 < COLS * kCh / 128; j0 += 8) {
    OUT y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = stage[(j0 + j) * 128 + row];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = ((j0 + j) * 128 + row) / kCh;
      if (i < left && c < room && in_bounds(to + i * width + c < end, status)) to[i * width + c] = y[j];
    }
  }
}

// The same as a call: in the loop over a pair's tiles, where nothing else waits for
// the writing warps, inlined it took 2048 x 4096 x 2001 from 26.9 us to 35, the
// products waiting with it.  Elsewhere the call costs more than it saves
// (40 x 4112 x 1001 on one CTA a tile: 15.6 us, inlined 15.3).
template <typename OUT, int kCh, int COLS>
__device__ __noinline__ void i8_copy_out_call(OUT *to, const OUT *stage, int64_t width, int left, int64_t room,
                                              const OUT *end, int row, int *status) {
  i8_copy_out<OUT, kCh, COLS>(to, stage, width, left, room, end, row, status);
}

// Writes COLS tokens of a tile's channels from the sums: four warps, a thread
// a channel (`row` of the tile, scale `ws`), tokens tok0 .. of the output with
// the scales xs[0 ..].  The outputs pass through shared memory, `buf` (two
// buffers, taken in turn), so that a token's channels leave in 16-byte pieces
// (as 2 bytes a lane they took three times as long).  Gated, rows 0..63 are the
// gates of rows 64..127: they give the later half of the tokens away and take
// the other rows' earlier half, and every thread computes half.
template <typename OUT, bool GATED, int COLS, bool PAIR>
__device__ __forceinline__ void i8_write(const I8Args &a, const uint32_t (&v)[COLS], float ws,
                                         const float *xs, int64_t tok0, int64_t ch0, int row, char *buf,
                                         int team) {
  constexpr int kCh = GATED ? 64 : 128, kPiece = 16 / sizeof(OUT);
  float *mail = reinterpret_cast<float *>(buf);
  OUT *stage = reinterpret_cast<OUT *>(buf + (GATED ? COLS * 64 * 4 : 0));
  // All loads from shared memory before any store, which might be to the same
  // place for all that the compiler knows, and no branch between activations:
  // one after the other they took a tile 15 us more.
  float y[COLS];
#pragma unroll
  for (int i = 0; i < COLS; ++i) y[i] = __uint_as_float(v[i]) * ws * xs[i];
  if constexpr (!GATED) {
#pragma unroll
    for (int i = 0; i < COLS; ++i) stage[i * kCh + row] = i8_out<OUT>(y[i]);
  } else {
    constexpr int kHalf = COLS / 2;
    const bool is_up = row >= 64;
    const int gives = is_up ? 0 : kHalf, first = is_up ? kHalf : 0;
    float kept[kHalf], other[kHalf];
#pragma unroll
    for (int i = 0; i < kHalf; ++i) {
      mail[(gives + i) * 64 + row % 64] = is_up ? y[i] : y[kHalf + i];
      kept[i] = is_up ? y[kHalf + i] : y[i];
    }
    i8_team_sync(team);
#pragma unroll
    for (int i = 0; i < kHalf; ++i) other[i] = mail[(first + i) * 64 + row % 64];
#pragma unroll
    for (int i = 0; i < kHalf; ++i)
      kept[i] = silu_mul(is_up ? other[i] : kept[i], is_up ? kept[i] : other[i]);
#pragma unroll
    for (int i = 0; i < kHalf; ++i) stage[(first + i) * kCh + row % 64] = i8_out<OUT>(kept[i]);
  }
  i8_team_sync(team);
  const int left = static_cast<int>(a.m - tok0 < COLS ? a.m - tok0 : COLS);
  OUT *to = static_cast<OUT *>(a.out) + tok0 * a.width + ch0;
  if (a.aligned) {
#pragma unroll
    for (int j = 0; j < COLS * kCh / kPiece / 128; ++j) {
      const int i = (j * 128 + row) / (kCh / kPiece), c = (j * 128 + row) % (kCh / kPiece) * kPiece;
      if (i < left && ch0 + c < a.width &&
          in_bounds((tok0 + i) * a.width + ch0 + c + kPiece <= a.m * a.width, a.status))
        *reinterpret_cast<uint4 *>(to + i * a.width + c) = *reinterpret_cast<const uint4 *>(stage + i * kCh + c);
    }
  } else {
    const OUT *end = static_cast<const OUT *>(a.out) + a.m * a.width;
    if constexpr (PAIR && !GATED)
      i8_copy_out_call<OUT, kCh, COLS>(to, stage, a.width, left, a.width - ch0, end, row, a.status);
    else
      i8_copy_out<OUT, kCh, COLS>(to, stage, a.width, left, a.width - ch0, end, row, a.status);
  }
  __syncwarp();  // behind stores that lanes skip: what comes next takes whole warps
}

// Where a wait gave up, before the cluster's last barrier: what its other CTAs send here
// lands first, parts (at `parts`, if any), which they send whether this CTA gave up or
// not, and arrivals that nobody waits for any more.
static __device__ __noinline__ void i8_settle(uint32_t parts, uint64_t settle_ns, int *status) {
  int never = 0;
  if (parts != 0) i8_wait(parts, 0, &never, settle_ns, status);
  __nanosleep(20000);
}

// Whether all of a team's warps are `fine`: a wait that one of them gave up ends
// all their parts in the barriers behind it.
#define ARN_I8_ALL_FINE(id)                                              \
  asm volatile(                                                          \
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"               \
      "barrier.cta.red.and.pred q, " #id ", 128, p;\n\t"                 \
      "selp.u32 %0, 1, 0, q;\n\t}"                                       \
      : "=r"(all)                                                        \
      : "r"(fine ? 1u : 0u)                                              \
      : "memory")
__device__ __forceinline__ bool i8_all_fine(bool fine, int team) {
  uint32_t all;
  if (team == 0)
    ARN_I8_ALL_FINE(1);
  else if (team == 1)
    ARN_I8_ALL_FINE(2);
  else if (team == 2)
    ARN_I8_ALL_FINE(3);
  else
    ARN_I8_ALL_FINE(4);
  return __all_sync(0xFFFFFFFFu, all != 0);
}
#undef ARN_I8_ALL_FINE

template <typename OUT, int NT, bool PAIR, bool GATED>
__global__ void __launch_bounds__(I8Shape<NT, PAIR>::kThreads, I8Shape<NT, PAIR>::kCtasPerSm)
    k_i8_tensor(const __grid_constant__ I8TensorArgs t) {
  using Shape = I8Shape<NT, PAIR>;
  constexpr int kGroup = PAIR ? 2 : 1;
  constexpr int kChannels = GATED ? 64 : 128;  // outputs' channels of a CTA's tile
  constexpr int kGroups = Shape::kTeams + 1;   // of four warps, of a pair's CTA
  constexpr bool kAllWrite = PAIR && GATED;    // groups that write a tile: write_tile
  constexpr int kWriters = kAllWrite ? kGroups : 1;
  extern __shared__ char smem_raw[];
  __shared__ I8Barriers bars;
  __shared__ float xs_of[NT], ws_of[128];
  const I8Args &a = t.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR || t.split > 1 ? cluster_ctarank() : 0;
  const uint32_t part = rank / kGroup, half = rank % kGroup;  // of the split, of a pair
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  float *const ring = reinterpret_cast<float *>(smem_raw + (base - smem_addr(smem_raw)));
  const uint32_t ops = base + Shape::kRaw * Shape::kRawBytes;
  volatile int *abort = &bars.abort;
  int *status = a.status;
  const uint64_t limit = t.waits.limit_ns;

  if (threadIdx.x == 0) {
    for (int i = 0; i < Shape::kRaw; ++i) {
      mbar_init(&bars.raw_full[i], 1);
      mbar_init(&bars.raw_empty[i], 4);
    }
    for (int i = 0; i < Shape::kOps; ++i) {
      mbar_init(&bars.op_full[i], 4 * kGroup);
      mbar_init(&bars.op_empty[i], 1);
    }
    mbar_init(&bars.acc_full, 1);
    mbar_init(&bars.acc_empty, 4 * kWriters * kGroup);
    mbar_init(&bars.parts, 1);
    mbar_init(&bars.quiet, 1);
    bars.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&t.w_map) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&t.x_map) : "memory");
  }
  // Before the next grid may start: the CTAs of one grid never wait for tensor
  // memory that the next one's hold.
  if (warp == 1) i8_tmem_alloc<PAIR>(smem_addr(&bars.tmem), Shape::kCols);

  // This CTA's k steps and tiles.
  const int steps = (a.K + kI8StepK - 1) / kI8StepK;
  const int step0 = steps * static_cast<int>(part) / t.split;
  const int step1 = steps * static_cast<int>(part + 1) / t.split;
  const int tiles = t.tiles_n * t.tiles_m;
  const int tile0 = static_cast<int>(blockIdx.x) / (kGroup * t.split);
  const int tile_step = static_cast<int>(gridDim.x) / (kGroup * t.split);
  const int my_tiles = (tiles - tile0 + tile_step - 1) / tile_step;
  const int total = my_tiles * (step1 - step0);  // stages
  // Tile -> (tile of channels, tile of tokens): pairs walk `group` token tiles
  // together over all channels, whose x then stays in L2.
  auto place = [&](int tile, int &tn, int &tm) {
    if constexpr (PAIR) {
      const int span = t.group * t.tiles_n;
      const int g = tile / span, rest = tile - g * span;
      const int width = min(t.group, t.tiles_m - g * t.group);
      tn = rest / width;
      tm = g * t.group + rest - tn * width;
    } else {
      tm = tile / t.tiles_n;
      tn = tile - tm * t.tiles_n;
    }
  };
  const uint32_t raw_full = smem_addr(bars.raw_full), raw_empty = smem_addr(bars.raw_empty);
  const uint32_t op_full = smem_addr(bars.op_full), op_empty = smem_addr(bars.op_empty);
  const uint32_t acc_full = smem_addr(&bars.acc_full), acc_empty = smem_addr(&bars.acc_empty);

  if (warp == 0 && i8_elect()) {
    // The first stages' weights, on their way to L2 while the previous grid ends.
    int tn, tm;
    place(tile0, tn, tm);
    const int ch = (tn * kGroup + static_cast<int>(half)) * kChannels;
    for (int s = step0; s < step1 && s < step0 + kI8Prefetch; ++s) {
      i8_prefetch_box(&t.w_map, s * kI8StepK, ch);
      i8_prefetch_box(&t.w_map, s * kI8StepK, GATED ? static_cast<int>(a.width) + ch : ch + 64);
    }
  }
  __syncwarp();

  i8_fence_before();
  if (PAIR || t.split > 1) {
    cluster_arrive_release();
    cluster_wait_acquire();
  }
  __syncthreads();
  i8_fence_after();
  const uint32_t tmem = bars.tmem;
  pdl_wait_prior_grid();
  pdl_launch_dependents();

  // The outputs of a pair's k-th tile, by group g.  Gated by all groups, a quarter of
  // the tokens each: the tensor cores wait until the sums have been read, and activations
  // take long (1792 x 4096 x 8192: 70.0 us, by the last group alone 72.9; 256 x 4096 x
  // 2002: 25.4 and 27.1).  Else by the last group: by all, rows of any width would wait
  // for one another's stores (8192 x 1024 x 4001: 68.8 us, by all 75.0; whole pieces
  // would gain, 2048 x 4096 x 2000: 25.5, by all 24.8).  False, for all of a group,
  // where a wait gave up or one was not `fine`.
  auto write_tile = [&](int k, int g, bool fine) -> bool {
    constexpr int kShare = NT / kWriters, kCols = kAllWrite ? 16 : 32;
    static_assert(!PAIR || kShare % kCols == 0, "whole chunks");
    static_assert(!kAllWrite || (kGroups * Shape::kBuffer / 2 <= Shape::kExchange &&
                                 16 * 64 * (4 + static_cast<int>(sizeof(OUT))) <= Shape::kBuffer / 2),
                  "a buffer for each group");
    int tn, tm;
    place(tile0 + k * tile_step, tn, tm);
    const int row = (warp & 3) * 32 + lane, first = kAllWrite ? g * kShare : 0;
    const int64_t ch0 = static_cast<int64_t>(tn * kGroup + static_cast<int>(half)) * kChannels;
    const int64_t ch = ch0 + (GATED ? row % 64 : row);
    const int64_t tok = static_cast<int64_t>(tm) * NT + first;
    const float ws = ch < a.width ? __ldg(a.ws + ch + (GATED && row >= 64 ? a.width : 0)) : 0.f;
#pragma unroll
    for (int i = 0; i < kShare; i += 128)
      if (i + row < kShare) xs_of[first + i + row] = tok + i + row < a.m ? __ldg(a.xs + tok + i + row) : 0.f;
    if (!i8_all_fine(fine && i8_wait(acc_full, static_cast<uint32_t>(k) & 1, abort, limit, status), g))
      return false;
    i8_fence_after();
    const uint32_t acc = tmem + (static_cast<uint32_t>(warp & 3) << 21) + first;
    // Gated, a group's chunks meet twice and need one buffer.
    char *buf = reinterpret_cast<char *>(ring) + Shape::kRings + (kAllWrite ? g * Shape::kBuffer / 2 : 0);
#pragma unroll 1
    for (int c = 0; c < kShare; c += kCols) {
      uint32_t v[kCols];
      if constexpr (kAllWrite)
        i8_tmem_load16(acc + c, v);
      else
        i8_tmem_load32(acc + c, v);
      if (c + kCols == kShare) {
        i8_fence_before();
        __syncwarp();
        if (lane == 0) i8_arrive_cluster(i8_mapa(acc_empty, rank & ~1u));
        __syncwarp();
      }
      i8_write<OUT, GATED, kCols, true>(a, v, ws, xs_of + first + c, tok + c, ch0, row,
                                        buf + (kAllWrite ? 0 : c / kCols % 2 * Shape::kBuffer), g);
    }
    return true;
  };

  if (warp == 0) {
    // ---- loads
    int r = 0, issued = 0;
    uint32_t phase = 0;
    bool fine = true;
    int end = step1;  // (a self-test stops a CTA before)
    if (t.waits.stop_rank < 0 || t.waits.stop_rank == static_cast<int>(rank))
      end = min(step1, step0 + t.waits.stop_after);
    for (int tile = tile0; fine && tile < tiles; tile += tile_step) {
      int tn, tm;
      place(tile, tn, tm);
      const int ch = (tn * kGroup + static_cast<int>(half)) * kChannels;
      const int ch2 = GATED ? static_cast<int>(a.width) + ch : ch + 64;
      const int tok = tm * NT + static_cast<int>(half) * Shape::kTokens;
      for (int s = step0; s < end; ++s) {
        fine = __all_sync(0xFFFFFFFFu, i8_wait(raw_empty + r * 8, phase ^ 1, abort, limit, status));
        if (!fine) break;
        // Checking build: the slot, and every stage within K.
        if (i8_elect() && in_bounds(r >= 0 && r < Shape::kRaw && s * kI8StepK < a.K, status)) {
          const uint32_t to = base + r * Shape::kRawBytes, bar = raw_full + r * 8;
          const int k = s * kI8StepK;
          mbar_arrive_expect_tx(&bars.raw_full[r], Shape::kRawBytes);
          i8_load_box(to, &t.w_map, k, ch, bar);
          i8_load_box(to + 64 * kI8StepK, &t.w_map, k, ch2, bar);
          i8_load_box(to + kI8RawW, &t.x_map, k, tok, bar);
        }
        if (issued < Shape::kRaw) ++issued;
        if (++r == Shape::kRaw) {
          r = 0;
          phase ^= 1;
        }
      }
      if (end < step1) break;
    }
    // Loads in flight land before this CTA's memory goes, whoever has given up.
    int never = 0;
#pragma unroll 1
    for (int i = 0; i < issued; ++i) {
      if (--r < 0) {
        r = Shape::kRaw - 1;
        phase ^= 1;
      }
      i8_wait(raw_full + r * 8, phase, &never, t.waits.settle_ns, status);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---- products
    if (half == 0) {
      // Instruction descriptor: fp32 sums, fp16 operands, both along k.
      constexpr uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(NT / 8) << 17) |
                                 (static_cast<uint32_t>(PAIR ? 16 : 8) << 24);
      // Shared-memory descriptor: 128-byte swizzle, 1024 bytes from eight rows
      // to the next eight.
      constexpr uint64_t kDesc = (uint64_t{2} << 61) | (uint64_t{1} << 46) | (uint64_t{64} << 32) |
                                 (uint64_t{1} << 16);
      int s = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool fine = true;
      for (int tile = tile0; fine && tile < tiles; tile += tile_step) {
        if (PAIR) {
          fine = __all_sync(0xFFFFFFFFu, i8_wait(acc_empty, acc_phase ^ 1, abort, limit, status));
          if (!fine) break;
        }
        for (int step = step0; step < step1; ++step) {
          fine = __all_sync(0xFFFFFFFFu, i8_wait(op_full + s * 8, phase, abort, limit, status));
          if (!fine) break;
          i8_fence_after();
          if (i8_elect()) {
            const uint32_t b = ops + s * Shape::kOpBytes;
            const uint32_t at = tmem + Shape::kAccCols + s * Shape::kOpCols;
#pragma unroll
            for (int ks = 0; ks < kI8StepK / 16; ++ks) {
              const uint32_t from = b + (ks >> 2) * (Shape::kTokens * 128) + (ks & 3) * 32;
              i8_mma<PAIR>(tmem, at + ks * 8, kDesc | ((from >> 4) & 0x3FFF), idesc,
                           step > step0 || ks > 0);
            }
            i8_commit<PAIR>(op_empty + s * 8, rank);
            if (step + 1 == step1) i8_commit<PAIR>(acc_full, rank);
          }
          __syncwarp();
          if (++s == Shape::kOps) {
            s = 0;
            phase ^= 1;
          }
        }
        if (fine) acc_phase ^= 1;
      }
      // Products in flight end before their operands and their sums go, whoever has
      // given up.
      int never = 0;
      if (i8_elect()) i8_commit_here<PAIR>(smem_addr(&bars.quiet));
      __syncwarp();
      i8_wait(smem_addr(&bars.quiet), 0, &never, t.waits.settle_ns, status);
    }
    __syncwarp();
  } else if (warp >= 4 && (kAllWrite || warp < Shape::kOutWarp0)) {
    // ---- operands: a team takes every kTeams-th stage; a thread unpacks a row
    // of w, and a row of x or a part of one (the lanes of a group of eight take
    // the same bytes of eight rows).
    const int team = (warp - 4) / 4, at = (warp & 3) * 32 + lane;
    const uint32_t a_lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21) + Shape::kAccCols;
    constexpr int kSets = 128 / Shape::kTokens;  // threads of a row of x
    constexpr int kChunks = 8 / kSets;
    static_assert(kSets >= 1 && kSets <= 8, "threads of a row of x");
    const int row = at % Shape::kTokens, set = at / Shape::kTokens;
    const uint32_t w_swizzle = at & 7, x_swizzle = row & 7;
    const uint32_t leader = PAIR ? i8_mapa(op_full, rank & ~1u) : 0;  // the CTA that issues the products
    int r = team, s = team;
    uint32_t raw_phase = 0, op_phase = 0;
    auto unpack = [&]() -> bool {
      if (!__all_sync(0xFFFFFFFFu, i8_wait(raw_full + r * 8, raw_phase, abort, limit, status))) return false;
      uint4 v[8], x[kChunks];
      const uint32_t raw = base + r * Shape::kRawBytes;
#pragma unroll
      for (uint32_t c = 0; c < 8; ++c) v[c] = i8_lds(raw + at * kI8StepK + ((c ^ w_swizzle) << 4));
#pragma unroll
      for (uint32_t c = 0; c < kChunks; ++c)
        x[c] = i8_lds(raw + kI8RawW + row * kI8StepK + (((set * kChunks + c) ^ x_swizzle) << 4));
      __syncwarp();
      if (lane == 0) i8_arrive(raw_empty + r * 8);
      if (!__all_sync(0xFFFFFFFFu, i8_wait(op_empty + s * 8, op_phase ^ 1, abort, limit, status))) return false;
      i8_fence_after();
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint32_t o[16];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          i8_unpack(v[h * 2 + c].x, o[c * 8], o[c * 8 + 1]);
          i8_unpack(v[h * 2 + c].y, o[c * 8 + 2], o[c * 8 + 3]);
          i8_unpack(v[h * 2 + c].z, o[c * 8 + 4], o[c * 8 + 5]);
          i8_unpack(v[h * 2 + c].w, o[c * 8 + 6], o[c * 8 + 7]);
        }
        i8_tmem_store16(a_lanes + s * Shape::kOpCols + h * 16, o);
      }
      const uint32_t to = ops + s * Shape::kOpBytes + row * 128;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const uint32_t chunk = set * kChunks + c, first = 2 * (chunk & 3);
        const uint32_t half = to + (chunk >> 2) * (Shape::kTokens * 128);
        uint32_t o[8];
        i8_unpack(x[c].x, o[0], o[1]);
        i8_unpack(x[c].y, o[2], o[3]);
        i8_unpack(x[c].z, o[4], o[5]);
        i8_unpack(x[c].w, o[6], o[7]);
        i8_sts(half + ((first ^ x_swizzle) << 4), o[0], o[1], o[2], o[3]);
        i8_sts(half + (((first + 1) ^ x_swizzle) << 4), o[4], o[5], o[6], o[7]);
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      i8_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR)
          i8_arrive_cluster(leader + s * 8);
        else
          i8_arrive(op_full + s * 8);
      }
      r += Shape::kTeams;
      if (r >= Shape::kRaw) {
        r -= Shape::kRaw;
        raw_phase ^= 1;
      }
      s += Shape::kTeams;
      if (s >= Shape::kOps) {
        s -= Shape::kOps;
        op_phase ^= 1;
      }
      return true;
    };
    if constexpr (!kAllWrite) {
      for (int n = team; n < total; n += Shape::kTeams)
        if (!unpack()) break;
    } else {
      // A tile is written behind the team's first stage of the next, which waits for
      // nothing but stages of tiles before; the last team only writes.  A warp whose
      // wait gave up goes on to its team's next tile, where the others learn of it.
      const int each = step1 - step0, to_write = t.split == 1 ? my_tiles : 0;
      bool fine = true;
      int n = team < Shape::kTeams ? team : total;
      for (int k = 0; k < to_write || (t.split > 1 && fine && n < total); n += Shape::kTeams) {
        if (fine && n < total) fine = unpack();
        bool all = true;
        while (all && k < to_write && (n >= total || n >= (k + 1) * each)) all = write_tile(k++, team, fine);
        if (!all) break;
      }
    }
    __syncwarp();
    if constexpr (!PAIR) {
      // ---- the sums: a thread a channel, 16 tokens a team in turn.  Every
      // stage has been read once they are done, and the rings are free.
      int tn, tm;
      place(tile0, tn, tm);
      const uint32_t acc = tmem + (static_cast<uint32_t>(warp & 3) << 21);
      const int64_t ch0 = static_cast<int64_t>(tn) * kChannels, ch = ch0 + (GATED ? at % 64 : at);
      const int64_t tok = static_cast<int64_t>(tm) * NT;
      const float ws = ch < a.width ? __ldg(a.ws + ch + (GATED && at >= 64 ? a.width : 0)) : 0.f;
      ws_of[at] = ws;  // each team the same
      if (at < NT) xs_of[at] = tok + at < a.m ? __ldg(a.xs + tok + at) : 0.f;
      const bool fine = i8_all_fine(i8_wait(acc_full, 0, abort, limit, status), team);
      if (t.split > 1) i8_cluster_arrive();  // this CTA's rings are free
      if (fine) {
        i8_fence_after();
#pragma unroll
        for (int c = 0; c < NT / 16; ++c) {
          if (c % Shape::kTeams != team) continue;
          uint32_t v[16];
          i8_tmem_load16(acc + c * 16, v);
          if (t.split == 1) {
            char *buf = reinterpret_cast<char *>(ring) +
                        (team * 2 + c / Shape::kTeams % 2) * Shape::kBuffer;
            i8_write<OUT, GATED, 16, false>(a, v, ws, xs_of + c * 16, tok + c * 16, ch0, at, buf, team);
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              ring[(c * 16 + i) * kI8TileRows + at] = __uint_as_float(v[i]);
          }
        }
        if (t.split > 1) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
    }
  } else if (PAIR && !kAllWrite && warp >= Shape::kOutWarp0 && t.split == 1) {
    for (int k = 0; k < my_tiles && write_tile(k, kGroups - 1, true);) ++k;
  }
  __syncwarp();
  if (PAIR && t.split > 1) {
    if (warp < 4) {
      i8_cluster_arrive();
      i8_cluster_wait();
    } else {
      // ---- outputs of a share of a tile's tokens: each pair of a split sends the
      // others their shares of its sums, keeps its own in tensor memory and adds
      // what comes, in the order of the parts.  All teams take part, 32 tokens
      // each in turn.
      static_assert(!PAIR || kGroups == 4, "i8_teams_sync");
      static_assert(!PAIR || NT < 256 || 2 * (NT / 2) * kI8TileRows * 4 + 2 * Shape::kBuffer <= Shape::kRings,
                    "buffers behind a split's sums");
      const int g = (warp - 4) / 4, row = (warp & 3) * 32 + lane;
      const uint32_t acc = tmem + (static_cast<uint32_t>(warp & 3) << 21), parts = smem_addr(&bars.parts);
      const int S = t.split, chunks = NT / 32 / S;  // of 32 tokens, of this CTA
      const int share = chunks * 32 * kI8TileRows;  // floats
      const float *inbox = ring + (S - 1) * share;
      int tn, tm;
      place(tile0, tn, tm);
      const int64_t ch0 = static_cast<int64_t>(tn * 2 + static_cast<int>(half)) * kChannels;
      const int64_t ch = ch0 + (GATED ? row % 64 : row);
      const int64_t tok = static_cast<int64_t>(tm) * NT;
      if (g == kGroups - 1) {  // idle until now: the others would wait for these
        ws_of[row] = ch < a.width ? __ldg(a.ws + ch + (GATED && row >= 64 ? a.width : 0)) : 0.f;
#pragma unroll
        for (int i = 0; i < NT; i += 128)
          if (i + row < NT) xs_of[i + row] = tok + i + row < a.m ? __ldg(a.xs + tok + i + row) : 0.f;
      }
      if (g == 0 && row == 0) mbar_arrive_expect_tx(&bars.parts, (S - 1) * share * 4);
      bool fine = i8_all_fine(i8_wait(acc_full, 0, abort, limit, status), g);
      i8_fence_after();
      i8_cluster_arrive();  // this CTA's rings are free
      for (int c = g; fine && c < NT / 32; c += kGroups) {
        const int to = c / chunks;
        if (to == static_cast<int>(part)) continue;
        float *out = ring + (to - (to > static_cast<int>(part))) * share +
                     (c - to * chunks) * 32 * kI8TileRows + row;
        if (!in_bounds(out + 31 * kI8TileRows < ring + (S - 1) * share, status)) continue;
        uint32_t v[32];
        i8_tmem_load32(acc + c * 32, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) out[i * kI8TileRows] = __uint_as_float(v[i]);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      i8_cluster_wait();  // those of all are
      i8_teams_sync();    // the sums to send are written, and the scales
      if (g == 0 && row < S - 1 && !*abort) {
        const uint32_t to = row + (row >= static_cast<int>(part));
        const uint32_t there = part - (part > to);
        asm volatile(
            "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
            ::"r"(i8_mapa(smem_addr(inbox + there * share), to * 2 + half)),
            "r"(smem_addr(ring + row * share)), "r"(share * 4), "r"(i8_mapa(parts, to * 2 + half))
            : "memory");
      }
      __syncwarp();
      if (g < chunks) {
        fine = i8_all_fine(fine && i8_wait(parts, 0, abort, limit, status), g);
        if (fine) {
          const int at = static_cast<int>(part) * chunks + g;
          uint32_t v[32];
          i8_tmem_load32(acc + at * 32, v);
          for (int p = 0; p < S - 1; ++p) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              v[i] = __float_as_uint(__uint_as_float(v[i]) +
                                     inbox[p * share + (g * 32 + i) * kI8TileRows + row]);
          }
          char *buf = reinterpret_cast<char *>(ring) +
                      (g < 2 ? Shape::kRings + g * Shape::kBuffer
                             : 2 * (S - 1) * share * 4 + (g - 2) * Shape::kBuffer);
          i8_write<OUT, GATED, 32, true>(a, v, ws_of[row], xs_of + at * 32, tok + at * 32, ch0, row, buf, g);
        }
      }
      if (!fine) i8_settle(parts, t.waits.settle_ns, status);
      __syncwarp();
    }
  }
  if (PAIR && warp == 1) {
    // Every arrival at this CTA that nobody has waited for comes before its
    // memory goes: of the last stages' products, of the last tile's readers.
    bool came = true;
    for (int i = 0; came && i < Shape::kOps && i < total; ++i) {
      const uint32_t n = static_cast<uint32_t>(total - 1 - i);
      came = i8_wait(op_empty + n % Shape::kOps * 8, n / Shape::kOps & 1, abort, limit, status);
    }
    if (came && half == 0 && t.split == 1)
      came = i8_wait(acc_empty, static_cast<uint32_t>(my_tiles - 1) & 1, abort, limit, status);
    if (!came) i8_settle(0, t.waits.settle_ns, status);
    __syncwarp();
  }

  if constexpr (!PAIR) {
    if (t.split > 1) {
      // ---- the parts of a tile: each CTA has its own [token][128 channels] in
      // its ring, and sends each CTA of the cluster that one's share of the
      // tokens, which sums them in the order of the ranks.
      const int S = t.split, cols = NT / S;
      const uint32_t share = static_cast<uint32_t>(cols) * kI8TileRows * 4;
      const uint32_t inbox = base + NT * kI8TileRows * 4, parts = smem_addr(&bars.parts);
      if (threadIdx.x == 0) mbar_arrive_expect_tx(&bars.parts, S * share);
      if (warp < 4) i8_cluster_arrive();
      i8_cluster_wait();  // the rings of all are free
      __syncthreads();    // the parts are written
      if (threadIdx.x < S && !*abort)
        asm volatile(
            "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
            ::"r"(i8_mapa(inbox + rank * share, threadIdx.x)), "r"(base + threadIdx.x * share), "r"(share),
            "r"(i8_mapa(parts, threadIdx.x))
            : "memory");
      int tn, tm;
      place(tile0, tn, tm);
      const int64_t ch0 = static_cast<int64_t>(tn) * kChannels;
      const int64_t tok0 = static_cast<int64_t>(tm) * NT + rank * cols;
      if (i8_wait(parts, 0, abort, limit, status)) {
        constexpr int kPiece = 16 / sizeof(OUT), kPieces = kChannels / kPiece;
        for (int i = threadIdx.x; i < cols * kPieces; i += Shape::kThreads) {
          const int col = i / kPieces, l = i % kPieces * kPiece;
          const float *from = ring + (NT + col) * kI8TileRows + l;
          float y[kPiece], up[kPiece];
#pragma unroll
          for (int e = 0; e < kPiece; ++e) y[e] = up[e] = 0.f;
          for (int p = 0; p < S; ++p, from += cols * kI8TileRows) {
#pragma unroll
            for (int e = 0; e < kPiece; e += 4) {
              const float4 f = *reinterpret_cast<const float4 *>(from + e);
              y[e] += f.x;
              y[e + 1] += f.y;
              y[e + 2] += f.z;
              y[e + 3] += f.w;
              if (GATED) {
                const float4 g = *reinterpret_cast<const float4 *>(from + 64 + e);
                up[e] += g.x;
                up[e + 1] += g.y;
                up[e + 2] += g.z;
                up[e + 3] += g.w;
              }
            }
          }
          const float xs = xs_of[rank * cols + col];
#pragma unroll
          for (int e = 0; e < kPiece; ++e) {
            y[e] = y[e] * ws_of[l + e] * xs;
            if (GATED) y[e] = silu_mul(y[e], up[e] * ws_of[64 + l + e] * xs);
          }
          if (tok0 + col >= a.m || !in_bounds(col < cols && l + kPiece <= kChannels, status)) continue;
          OUT *to = static_cast<OUT *>(a.out) + (tok0 + col) * a.width + ch0 + l;
          if (a.aligned) {
            if (ch0 + l < a.width) *reinterpret_cast<uint4 *>(to) = i8_pack<OUT>(y);
          } else {
#pragma unroll
            for (int e = 0; e < kPiece; ++e)
              if (ch0 + l + e < a.width) to[e] = i8_out<OUT>(y[e]);
          }
        }
      } else {
        i8_settle(parts, t.waits.settle_ns, status);
      }
      __syncwarp();
    }
  }
  // Nobody leaves while its cluster may still use its memory.
  i8_fence_before();
  if (PAIR || t.split > 1) {
    i8_cluster_arrive();
    i8_cluster_wait();
  }
  __syncthreads();
  i8_fence_after();
  if (warp == 1) i8_tmem_free<PAIR>(tmem, Shape::kCols);
}

using I8TensorKernel = void (*)(I8TensorArgs);

struct I8Tensor {
  I8TensorKernel kernel;
  int threads, smem, x_rows;
};

template <typename OUT, int NT, bool PAIR>
inline I8Tensor i8_tensor_one(bool gated) {
  using Shape = I8Shape<NT, PAIR>;
  return {gated ? &k_i8_tensor<OUT, NT, PAIR, true> : &k_i8_tensor<OUT, NT, PAIR, false>, Shape::kThreads,
          Shape::kSmem, Shape::kTokens};
}

// tokens: 16 or 32 of one CTA, 64, 128 or 256 of a pair.
template <typename OUT>
inline I8Tensor i8_tensor_of(int tokens, bool pair, bool gated) {
  if (pair)
    return tokens == 64    ? i8_tensor_one<OUT, 64, true>(gated)
           : tokens == 128 ? i8_tensor_one<OUT, 128, true>(gated)
                           : i8_tensor_one<OUT, 256, true>(gated);
  return tokens == 16 ? i8_tensor_one<OUT, 16, false>(gated) : i8_tensor_one<OUT, 32, false>(gated);
}

I8Tensor i8_tensor_f32(int tokens, bool pair, bool gated);
I8Tensor i8_tensor_bf16(int tokens, bool pair, bool gated);
I8Tensor i8_tensor_f16(int tokens, bool pair, bool gated);

}  // namespace arn
