#include "block_norm.cuh"

namespace arn {

BlockNormKernel block_norm_f16(bool r32, bool cluster, int threads, int *ctas) {
  return block_norm_of<__half>(r32, cluster, threads, ctas);
}

}  // namespace arn
