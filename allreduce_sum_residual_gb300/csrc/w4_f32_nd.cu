// The 4-bit products' kernels (w4_matvec.cuh) with f32 scales, no zero points,
// one matrix: apart from the others so that they compile in parallel.
#include "w4_matvec.cuh"

namespace arn {

W4Kernel w4_kernel_f32_nd(int r, int nt, int group) {
  return w4_pick<AR_TYPE_F32, false, false>(r, nt, group);
}

}  // namespace arn
