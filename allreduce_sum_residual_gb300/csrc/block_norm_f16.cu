#include "block_norm.cuh"

namespace arn {

BlockNormKernel block_norm_f16(bool r32, bool cluster, int vpt, int *registers) {
  return block_norm_of<__half>(r32, cluster, vpt, registers);
}

}  // namespace arn
