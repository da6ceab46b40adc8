// Products of 8-bit integers with scales for each token and channel
// (ar_i8_matmul): the kernels' arguments and what they share.
//
//   out[i, j] = xs_i ws_j sum_k x[i, k] w[j, k],  or its gated half
#pragma once

#include "dense.cuh"

namespace arn {

struct I8Args {
  const int8_t *x;   // [m, K]
  const float *xs;   // [m]
  const int8_t *w;   // [N, K]
  const float *ws;   // [N]
  void *out;         // [m, width] of out_type
  int64_t m, width;  // width: N, or N / 2 with the gated activation
  int N, K;
  int gated, out_type;
  int aligned;       // tensor cores: rows of out start and end at 16 bytes
  int team;          // matvec: warps of a row block
  int token_blocks;  // matvec: CTAs beside one another for the tokens
  int *status;
};

__device__ __forceinline__ void i8_store(const I8Args &a, int64_t at, float v) {
  if (a.out_type == AR_TYPE_F32)
    static_cast<float *>(a.out)[at] = v;
  else if (a.out_type == AR_TYPE_BF16)
    static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(v);
  else
    static_cast<__half *>(a.out)[at] = __float2half_rn(v);
}

// gate / (1 + exp(-gate)) * up; the reciprocal is within a step (of any
// divisor up to infinity, where it is 0).
__device__ __forceinline__ float silu_mul(float gate, float up) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.f + expf(-gate)));
  return gate * r * up;
}

cudaError_t launch_i8_matvec(I8Args a, int sms, cudaStream_t stream);
struct I8Plan {
  int tokens;  // of a tile: 16 or 32 of one CTA, 64, 128 or 256 of a pair; 0: matvec
  int split;   // parts of K
  bool pair;
};
// How long the tensor kernels' waits may take before they give up, and after that
// those for what is still under way to a CTA; for the self-test a rank of the
// cluster (-1: all) that loads no more than so many stages.
constexpr int kI8AllStages = 1 << 20;  // more than AR_I8_MAX_K has
struct I8Waits {
  uint64_t limit_ns, settle_ns;
  int stop_rank, stop_after;
};
// `pairs`: that run at a time.  An AR_* status.
int launch_i8_tensor(const I8Args &a, const I8Plan &plan, int pairs, cudaStream_t stream,
                     const I8Waits *waits = nullptr);
// Shared memory for the tensor kernels, once per device, and the clusters of 1, 2
// and 4 pairs that the current device runs at a time.
int ready_i8_tensor(int sms, const int **pairs);

}  // namespace arn
