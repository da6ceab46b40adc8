// Products of 8-bit integers on the tensor cores (ar_i8_matmul above a few
// tokens): the kernel.
//
// The part's own 8-bit integer rate is far below its 16-bit floating-point
// rate, so the bytes are multiplied as fp16: every byte is exact there, a
// product of two has 14 bits, and fp32 adds whole numbers exactly up to 2^24.
//
// The tile.  The weights' rows are the 128 rows of the accumulator (256 of a
// pair of CTAs, each holding its own 128), the tokens its columns.  So one
// kernel serves from 16 tokens, where the weights' bytes are the bound and
// each is read once, to prompts, where the tensor cores are.  Lane l of tensor
// memory is a channel, and a warp's stores of one token are 32 channels in a
// row.
//
// The operands are unpacked on the way.  TMA brings boxes of 64 rows x 128
// bytes of w and TB x 128 of x (128-byte swizzle; what lies behind the arrays'
// ends comes as zeros, which add nothing).  Four warps turn the tile of w into
// fp16 in tensor memory, from where the tensor core takes its A operand: a
// thread is a row, as in tensor memory, so unpacked weights, twice the bytes,
// never pass through shared memory.  The others turn x into the swizzled fp16
// tile of the B operand.  A byte b becomes 1024 + (b + 128) by a byte
// permutation under the exponent of 1024, and one half2 subtraction leaves b
// (a published method: Kim, Henry, Fahim and Awadalla, "Who Says Elephants
// Can't Run", 2022).
//
// Roles: a thread issues the loads, a thread the products, four warps unpack
// w, some unpack x, and of a pair four more write the outputs while the next
// tile's operands are unpacked.  Between them rings of mbarriers, every wait
// bounded.  A pair of CTAs is persistent and takes tiles in turn; one CTA
// takes one tile, or with few tiles a cluster of `split` CTAs takes one, each
// a part of K, and adds the parts up through the cluster's shared memory in
// the order of their ranks.
#pragma once

#include <cuda.h>

#include "i8_matmul.cuh"

namespace arn {

struct I8TensorArgs {
  CUtensorMap w_map, x_map;
  I8Args a;
  int tiles_n, tiles_m;  // tiles of channels, of tokens
  int split;             // CTAs of a tile (one CTA a tile)
  int group;             // token tiles that are walked together (pairs)
  uint64_t wait_limit_ns;
};

constexpr int kI8TileRows = 128;  // channels of a CTA
constexpr int kI8StepK = 128;     // k of a stage
constexpr int kI8RawW = kI8TileRows * kI8StepK;

// NT: tokens of a tile; PAIR: two CTAs share it.
template <int NT, bool PAIR>
struct I8Shape {
  static constexpr int kTokens = PAIR ? NT / 2 : NT;  // tokens whose x this CTA holds
  static constexpr int kXWarps = kTokens <= 64 ? 2 : 4;
  static constexpr int kXWarp0 = kXWarps == 2 ? 2 : 8;
  static constexpr int kWarps = PAIR ? 16 : kXWarps == 2 ? 8 : 12;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kOps = PAIR || NT <= 32 ? 3 : 2;  // stages of unpacked operands
  static constexpr int kRaw = PAIR ? 3 : NT <= 16 ? 5 : NT <= 32 ? 4 : NT <= 64 ? 3 : 4;
  static constexpr int kRawX = kTokens * kI8StepK;
  static constexpr int kRawBytes = kI8RawW + kRawX;
  static constexpr int kOpBytes = kTokens * kI8StepK * 2;
  static constexpr int kAccCols = NT < 32 ? 32 : NT;
  static constexpr int kOpCols = kI8StepK / 2;
  static constexpr int kCols = kAccCols + kOps * kOpCols <= 256 ? 256 : 512;
  static constexpr int kExchange = PAIR ? 2 * 2 * 16 * 64 * 4 : 0;
  // One CTA a tile: the parts of a tile, in the rings' place.
  static constexpr int kRings = kRaw * kRawBytes + kOps * kOpBytes;
  static constexpr int kSmem = 1024 + kRings + kExchange;
  static constexpr int kCtasPerSm = kCols == 256 && kSmem <= 113 * 1024 ? 2 : 1;
  static_assert(PAIR || NT * kI8TileRows * 4 <= kRings, "the parts of a tile fit the rings");
  static_assert(kSmem <= 230 * 1024 - 512, "shared memory of a CTA");
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
// arrive at.
__device__ __forceinline__ bool i8_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                        uint64_t limit_ns, int *status) {
  if (i8_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (i8_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      *abort_flag = 1;
      if (status) atomicExch(status, AR_ERR_TIMEOUT);
      return false;
    }
  }
}

__device__ __forceinline__ uint32_t i8_mapa(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void i8_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void i8_arrive_cluster(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
               : "memory");
}

__device__ __forceinline__ void i8_load_box(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar)
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

// Arrives at `bar` (of both CTAs of a pair) once this thread's products so far
// are done.
template <bool PAIR>
__device__ __forceinline__ void i8_commit(uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(bar), "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}

__device__ __forceinline__ void i8_tmem_store32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
      "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
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
  uint64_t raw_full[8], raw_empty[8], op_full[4], op_empty[4], acc_full, acc_empty;
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

template <typename OUT, int NT, bool PAIR, bool GATED>
__global__ void __launch_bounds__(I8Shape<NT, PAIR>::kThreads, I8Shape<NT, PAIR>::kCtasPerSm)
    k_i8_tensor(const __grid_constant__ I8TensorArgs t) {
  using Shape = I8Shape<NT, PAIR>;
  constexpr int kGroup = PAIR ? 2 : 1;
  constexpr int kChannels = GATED ? 64 : 128;  // outputs' channels of a CTA's tile
  extern __shared__ char smem_raw[];
  __shared__ I8Barriers bars;
  const I8Args &a = t.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR || t.split > 1 ? cluster_ctarank() : 0;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t ops = base + Shape::kRaw * Shape::kRawBytes;
  volatile int *abort = &bars.abort;
  int *status = a.status;
  const uint64_t limit = t.wait_limit_ns;

  constexpr int kUnpackers = 4 + Shape::kXWarps;
  if (threadIdx.x == 0) {
    for (int i = 0; i < Shape::kRaw; ++i) {
      mbar_init(&bars.raw_full[i], 1);
      mbar_init(&bars.raw_empty[i], kUnpackers);
    }
    for (int i = 0; i < Shape::kOps; ++i) {
      mbar_init(&bars.op_full[i], kUnpackers * kGroup);
      mbar_init(&bars.op_empty[i], 1);
    }
    mbar_init(&bars.acc_full, 1);
    mbar_init(&bars.acc_empty, 4 * kGroup);
    bars.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&t.w_map) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&t.x_map) : "memory");
  }
  // Before the next grid may start: the CTAs of one grid never wait for tensor
  // memory that the next one's hold.
  if (warp == 1) i8_tmem_alloc<PAIR>(smem_addr(&bars.tmem), Shape::kCols);
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

  // This CTA's k steps and tiles.
  const int steps = (a.K + kI8StepK - 1) / kI8StepK;
  int step0 = 0, step1 = steps;
  if (!PAIR) {
    step0 = static_cast<int>(static_cast<int64_t>(steps) * rank / t.split);
    step1 = static_cast<int>(static_cast<int64_t>(steps) * (rank + 1) / t.split);
  }
  const int64_t tiles = static_cast<int64_t>(t.tiles_n) * t.tiles_m;
  const int64_t tile0 = PAIR ? blockIdx.x / 2 : blockIdx.x / t.split;
  const int64_t tile_step = PAIR ? gridDim.x / 2 : tiles;
  // Tile -> (tile of channels, tile of tokens): pairs walk `group` token tiles
  // together over all channels, whose x then stays in L2.
  auto place = [&](int64_t tile, int &tn, int &tm) {
    if constexpr (PAIR) {
      const int64_t span = static_cast<int64_t>(t.group) * t.tiles_n;
      const int g = static_cast<int>(tile / span);
      const int rest = static_cast<int>(tile - g * span);
      const int width = min(t.group, t.tiles_m - g * t.group);
      tm = g * t.group + rest % width;
      tn = rest / width;
    } else {
      tn = static_cast<int>(tile % t.tiles_n);
      tm = static_cast<int>(tile / t.tiles_n);
    }
  };

  const uint32_t raw_full = smem_addr(bars.raw_full), raw_empty = smem_addr(bars.raw_empty);
  const uint32_t op_full = smem_addr(bars.op_full), op_empty = smem_addr(bars.op_empty);
  const uint32_t acc_full = smem_addr(&bars.acc_full), acc_empty = smem_addr(&bars.acc_empty);

  if (warp == 0) {
    // ---- loads
    if (lane == 0) {
      int r = 0, issued = 0;
      uint32_t phase = 0;
      bool fine = true;
      for (int64_t tile = tile0; fine && tile < tiles; tile += tile_step) {
        int tn, tm;
        place(tile, tn, tm);
        const int ch = (PAIR ? tn * 2 + static_cast<int>(rank) : tn) * kChannels;
        const int tok = tm * NT + (PAIR ? static_cast<int>(rank) * Shape::kTokens : 0);
        for (int s = step0; s < step1; ++s) {
          fine = i8_wait(raw_empty + r * 8, phase ^ 1, abort, limit, status);
          if (!fine) break;
          const uint32_t to = base + r * Shape::kRawBytes, bar = raw_full + r * 8;
          mbar_arrive_expect_tx(&bars.raw_full[r], Shape::kRawBytes);
          const int k = s * kI8StepK;
          i8_load_box(to, &t.w_map, k, ch, bar);
          i8_load_box(to + 64 * kI8StepK, &t.w_map, k, GATED ? static_cast<int>(a.width) + ch : ch + 64,
                      bar);
          i8_load_box(to + kI8RawW, &t.x_map, k, tok, bar);
          if (issued < Shape::kRaw) ++issued;
          if (++r == Shape::kRaw) {
            r = 0;
            phase ^= 1;
          }
        }
      }
      if (!fine) {
        // Loads in flight land before this CTA's memory goes.
        int never = 0;
        for (int i = 0; i < issued; ++i) {
          if (--r < 0) {
            r = Shape::kRaw - 1;
            phase ^= 1;
          }
          i8_wait(raw_full + r * 8, phase, &never, limit, status);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---- products
    if (lane == 0 && rank % kGroup == 0) {
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
      for (int64_t tile = tile0; fine && tile < tiles; tile += tile_step) {
        if (PAIR) {
          fine = i8_wait(acc_empty, acc_phase ^ 1, abort, limit, status);
          if (!fine) break;
          i8_fence_after();
        }
        for (int step = step0; step < step1; ++step) {
          fine = i8_wait(op_full + s * 8, phase, abort, limit, status);
          if (!fine) break;
          i8_fence_after();
          const uint32_t b = ops + s * Shape::kOpBytes;
          const uint32_t at = tmem + Shape::kAccCols + s * Shape::kOpCols;
#pragma unroll
          for (int ks = 0; ks < kI8StepK / 16; ++ks) {
            const uint32_t from = b + (ks >> 2) * (Shape::kTokens * 128) + (ks & 3) * 32;
            i8_mma<PAIR>(tmem, at + ks * 8, kDesc | ((from >> 4) & 0x3FFF), idesc,
                         step > step0 || ks > 0);
          }
          i8_commit<PAIR>(op_empty + s * 8);
          if (++s == Shape::kOps) {
            s = 0;
            phase ^= 1;
          }
        }
        if (fine) {
          i8_commit<PAIR>(acc_full);
          acc_phase ^= 1;
        }
      }
      if (!fine) {
        // Products in flight end before their operands go.
        int never = 0;
        i8_commit<PAIR>(acc_full);
        i8_wait(acc_full, acc_phase, &never, limit, status);
      }
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 8) {
    // ---- w: a thread a row
    const int row = (warp - 4) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(warp - 4) << 21;  // 32 lanes a warp
    const uint32_t leader = PAIR ? i8_mapa(op_full, 0) : 0;
    int r = 0, s = 0;
    uint32_t raw_phase = 0, op_phase = 0;
    bool fine = true;
    for (int64_t tile = tile0; fine && tile < tiles; tile += tile_step) {
      for (int step = step0; step < step1; ++step) {
        fine = i8_wait(raw_full + r * 8, raw_phase, abort, limit, status);
        if (!__all_sync(0xFFFFFFFFu, fine)) {
          fine = false;
          break;
        }
        uint4 v[8];
        const uint32_t from = base + r * Shape::kRawBytes + row * kI8StepK;
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = i8_lds(from + ((c ^ (row & 7)) << 4));
        __syncwarp();
        if (lane == 0) i8_arrive(raw_empty + r * 8);
        fine = i8_wait(op_empty + s * 8, op_phase ^ 1, abort, limit, status);
        if (!__all_sync(0xFFFFFFFFu, fine)) {
          fine = false;
          break;
        }
        i8_fence_after();
        const uint32_t at = tmem + lanes + Shape::kAccCols + s * Shape::kOpCols;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t o[32];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            i8_unpack(v[h * 4 + c].x, o[c * 8], o[c * 8 + 1]);
            i8_unpack(v[h * 4 + c].y, o[c * 8 + 2], o[c * 8 + 3]);
            i8_unpack(v[h * 4 + c].z, o[c * 8 + 4], o[c * 8 + 5]);
            i8_unpack(v[h * 4 + c].w, o[c * 8 + 6], o[c * 8 + 7]);
          }
          i8_tmem_store32(at + h * 32, o);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        i8_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR)
            i8_arrive_cluster(leader + s * 8);
          else
            i8_arrive(op_full + s * 8);
        }
        if (++r == Shape::kRaw) {
          r = 0;
          raw_phase ^= 1;
        }
        if (++s == Shape::kOps) {
          s = 0;
          op_phase ^= 1;
        }
      }
    }
  } else if (warp >= Shape::kXWarp0 && warp < Shape::kXWarp0 + Shape::kXWarps) {
    // ---- x: the lanes of a group of eight take eight rows' same bytes
    constexpr int kThreadsX = Shape::kXWarps * 32;
    constexpr int kSets = kThreadsX / Shape::kTokens;  // threads of a row
    constexpr int kChunks = 8 / kSets;
    static_assert(kSets >= 1 && kSets <= 8, "threads of a row");
    const int at = (warp - Shape::kXWarp0) * 32 + lane;
    const int row = at % Shape::kTokens, set = at / Shape::kTokens;
    const uint32_t leader = PAIR ? i8_mapa(op_full, 0) : 0;
    int r = 0, s = 0;
    uint32_t raw_phase = 0, op_phase = 0;
    bool fine = true;
    for (int64_t tile = tile0; fine && tile < tiles; tile += tile_step) {
      for (int step = step0; step < step1; ++step) {
        fine = i8_wait(raw_full + r * 8, raw_phase, abort, limit, status);
        if (!__all_sync(0xFFFFFFFFu, fine)) {
          fine = false;
          break;
        }
        uint4 v[kChunks];
        const uint32_t from = base + r * Shape::kRawBytes + kI8RawW + row * kI8StepK;
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          v[c] = i8_lds(from + (((set * kChunks + c) ^ (row & 7)) << 4));
        __syncwarp();
        if (lane == 0) i8_arrive(raw_empty + r * 8);
        fine = i8_wait(op_empty + s * 8, op_phase ^ 1, abort, limit, status);
        if (!__all_sync(0xFFFFFFFFu, fine)) {
          fine = false;
          break;
        }
        const uint32_t to = ops + s * Shape::kOpBytes + row * 128;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          const int chunk = set * kChunks + c;
          const uint32_t half = to + (chunk >> 2) * (Shape::kTokens * 128);
          const uint32_t first = 2 * (chunk & 3);
          uint32_t o[8];
          i8_unpack(v[c].x, o[0], o[1]);
          i8_unpack(v[c].y, o[2], o[3]);
          i8_unpack(v[c].z, o[4], o[5]);
          i8_unpack(v[c].w, o[6], o[7]);
          i8_sts(half + ((first ^ (row & 7)) << 4), o[0], o[1], o[2], o[3]);
          i8_sts(half + (((first + 1) ^ (row & 7)) << 4), o[4], o[5], o[6], o[7]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          if (PAIR)
            i8_arrive_cluster(leader + s * 8);
          else
            i8_arrive(op_full + s * 8);
        }
        if (++r == Shape::kRaw) {
          r = 0;
          raw_phase ^= 1;
        }
        if (++s == Shape::kOps) {
          s = 0;
          op_phase ^= 1;
        }
      }
    }
  } else if (PAIR && warp >= 12) {
    // ---- outputs of a pair's tile: a thread a channel
    const int q = warp - 12, row = q * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(q) << 21;
    const uint32_t leader_empty = i8_mapa(acc_empty, 0);
    float *exchange = reinterpret_cast<float *>(smem_raw + (base - smem_addr(smem_raw)) + Shape::kRings);
    OUT *out = static_cast<OUT *>(a.out);
    uint32_t acc_phase = 0;
    for (int64_t tile = tile0; tile < tiles; tile += tile_step) {
      int tn, tm;
      place(tile, tn, tm);
      const int64_t ch = static_cast<int64_t>(tn * 2 + static_cast<int>(rank)) * kChannels +
                         (GATED ? row % 64 : row);
      const int64_t tok = static_cast<int64_t>(tm) * NT;
      const bool mine = ch < a.width;
      const float ws = mine ? __ldg(a.ws + ch + (GATED && row >= 64 ? a.width : 0)) : 0.f;
      bool fine = i8_wait(acc_full, acc_phase, abort, limit, status);
      if (GATED) {  // the four warps meet below: all go on or none
        uint32_t all;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
            "barrier.cta.red.and.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
            : "=r"(all)
            : "r"(fine ? 1u : 0u)
            : "memory");
        fine = all != 0;
      }
      if (!__all_sync(0xFFFFFFFFu, fine)) break;
      acc_phase ^= 1;
      i8_fence_after();
#pragma unroll 1
      for (int cb = 0; cb < NT / 32; ++cb) {
        uint32_t v[32];
        i8_tmem_load32(tmem + lanes + cb * 32, v);
        if (cb == NT / 32 - 1) {
          i8_fence_before();
          __syncwarp();
          if (lane == 0) i8_arrive_cluster(leader_empty);
        }
        const int64_t tok0 = tok + cb * 32;
        const int left = static_cast<int>(a.m - tok0 < 32 ? a.m - tok0 : 32);
        const float xs = lane < left ? __ldg(a.xs + tok0 + lane) : 0.f;
        OUT *to = out + tok0 * a.width + ch;
        if constexpr (!GATED) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float y = __uint_as_float(v[i]) * ws * __shfl_sync(0xFFFFFFFFu, xs, i);
            if (mine && i < left) to[i * a.width] = i8_out<OUT>(y);
          }
        } else {
          // Gate rows give the later 16 tokens away and take the up rows'
          // earlier 16, so that every thread writes half.
          const bool is_up = row >= 64;
          float *mail = exchange + (cb & 1) * (2 * 16 * 64);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float y = __uint_as_float(v[i]) * ws * __shfl_sync(0xFFFFFFFFu, xs, i);
            v[i] = __float_as_uint(y);
            if (is_up == (i < 16)) mail[((is_up ? 0 : 16) + i % 16) * 64 + row % 64] = y;
          }
          asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int at = is_up ? 16 + i : i;
            const float other = mail[at * 64 + row % 64];
            const float mine_v = __uint_as_float(is_up ? v[16 + i] : v[i]);
            const float y = is_up ? silu_mul(other, mine_v) : silu_mul(mine_v, other);
            if (mine && at < left) to[at * a.width] = i8_out<OUT>(y);
          }
        }
      }
    }
  }
  __syncwarp();

  if constexpr (!PAIR) {
    // ---- outputs of one CTA's tile, or of its part of the tokens: the parts
    // [rank][token][128 channels] of a tile's split, in rank order.
    int tn, tm;
    place(tile0, tn, tm);
    const int S = t.split, cols = NT / S;
    bool fine = true;
    if (warp >= 4 && warp < 8) {
      fine = i8_wait(acc_full, 0, abort, limit, status);
      fine = __all_sync(0xFFFFFFFFu, fine);
      i8_fence_after();
    }
    // Every CTA's rings are idle.
    if (S > 1) {
      cluster_arrive_release();
      cluster_wait_acquire();
    } else {
      __syncthreads();
    }
    if (warp >= 4 && warp < 8 && fine) {
      const uint32_t lanes = static_cast<uint32_t>(warp - 4) << 21;
      const uint32_t row = base + ((warp - 4) * 32 + lane) * 4;
#pragma unroll 1
      for (int c0 = 0; c0 < NT; c0 += 16) {
        uint32_t v[16];
        i8_tmem_load16(tmem + lanes + c0, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int owner = (c0 + i) / cols, col = (c0 + i) % cols;
          const uint32_t at = row + (rank * cols + col) * (kI8TileRows * 4);
          if (S > 1)
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(i8_mapa(at, owner)), "r"(v[i])
                         : "memory");
          else
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(v[i]) : "memory");
        }
      }
    }
    if (S > 1) {
      cluster_arrive_release();
      cluster_wait_acquire();
    } else {
      __syncthreads();
    }
    const float *parts =
        reinterpret_cast<const float *>(smem_raw + (base - smem_addr(smem_raw)));
    OUT *out = static_cast<OUT *>(a.out);
    const int64_t ch0 = static_cast<int64_t>(tn) * kChannels;
    const int64_t tok0 = static_cast<int64_t>(tm) * NT + rank * cols;
    if (!bars.abort) {
      for (int i = threadIdx.x; i < cols * kChannels; i += Shape::kThreads) {
        const int l = i % kChannels, col = i / kChannels;
        const int64_t ch = ch0 + l, tok = tok0 + col;
        if (ch >= a.width || tok >= a.m) continue;
        float y = 0.f, up = 0.f;
        for (int p = 0; p < S; ++p) {
          const float *from = parts + (p * cols + col) * kI8TileRows + l;
          y += from[0];
          if (GATED) up += from[64];
        }
        const float xs = __ldg(a.xs + tok);
        y = y * __ldg(a.ws + ch) * xs;
        if (GATED) y = silu_mul(y, up * __ldg(a.ws + ch + a.width) * xs);
        out[tok * a.width + ch] = i8_out<OUT>(y);
      }
    }
  }
  // Nobody leaves while its pair may still use its memory.
  i8_fence_before();
  if (PAIR) {
    cluster_arrive_release();
    cluster_wait_acquire();
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

// tokens: 16, 32, 64 or 128 of one CTA, 256 of a pair.
template <typename OUT>
inline I8Tensor i8_tensor_of(int tokens, bool gated) {
  switch (tokens) {
    case 16: return i8_tensor_one<OUT, 16, false>(gated);
    case 32: return i8_tensor_one<OUT, 32, false>(gated);
    case 64: return i8_tensor_one<OUT, 64, false>(gated);
    case 128: return i8_tensor_one<OUT, 128, false>(gated);
    default: return i8_tensor_one<OUT, 256, true>(gated);
  }
}

I8Tensor i8_tensor_f32(int tokens, bool gated);
I8Tensor i8_tensor_bf16(int tokens, bool gated);
I8Tensor i8_tensor_f16(int tokens, bool gated);

}  // namespace arn
