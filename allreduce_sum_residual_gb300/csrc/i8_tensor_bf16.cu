#include "i8_tensor.cuh"

namespace arn {

I8Tensor i8_tensor_bf16(int tokens, bool pair, bool gated) {
  return i8_tensor_of<__nv_bfloat16>(tokens, pair, gated);
}

}  // namespace arn
