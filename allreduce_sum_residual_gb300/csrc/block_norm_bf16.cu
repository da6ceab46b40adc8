#include "block_norm.cuh"

namespace arn {

BlockNormKernel block_norm_bf16(bool r32, bool cluster, int threads, int *ctas) {
  return block_norm_of<__nv_bfloat16>(r32, cluster, threads, ctas);
}

}  // namespace arn
