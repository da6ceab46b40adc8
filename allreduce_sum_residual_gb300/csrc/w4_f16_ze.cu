// The 4-bit products' kernels (w4_matvec.cuh) with f16 scales, zero points,
// the routed experts: apart from the others so that they compile in parallel.
#include "w4_matvec.cuh"

namespace arn {

W4Kernel w4_kernel_f16_ze(int r, int nt, int group) {
  return w4_pick<AR_TYPE_F16, true, true>(r, nt, group);
}

}  // namespace arn
