#include "i8_tensor.cuh"

namespace arn {

I8Tensor i8_tensor_f32(int tokens, bool pair, bool gated) {
  return i8_tensor_of<float>(tokens, pair, gated);
}

}  // namespace arn
