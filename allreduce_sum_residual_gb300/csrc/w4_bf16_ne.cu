// The 4-bit products' kernels (w4_matvec.cuh) with bf16 scales, no zero points,
// the routed experts: apart from the others so that they compile in parallel.
#include "w4_matvec.cuh"

namespace arn {

W4Kernel w4_kernel_bf16_ne(int r, int nt, int group) {
  return w4_pick<AR_TYPE_BF16, false, true>(r, nt, group);
}

}  // namespace arn
