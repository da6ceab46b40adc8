#include "i8_tensor.cuh"

namespace arn {

I8Tensor i8_tensor_f16(int tokens, bool pair, bool gated) {
  return i8_tensor_of<__half>(tokens, pair, gated);
}

}  // namespace arn
