#include "block_norm.cuh"

namespace arn {

BlockNormKernel block_norm_bf16(bool r32, bool cluster, int vpt, int *registers) {
  return block_norm_of<__nv_bfloat16>(r32, cluster, vpt, registers);
}

}  // namespace arn
