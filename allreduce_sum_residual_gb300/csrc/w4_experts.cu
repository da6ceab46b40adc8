// ar_w4_matvec_experts' kernels (see w4_matvec.cuh), in a translation unit of
// their own so that they compile beside the dense ones.
#include "w4_matvec.cuh"

namespace arn {

W4Kernel w4_experts_kernel(int r, int nt, int group) { return w4_pick<true>(r, nt, group); }

}  // namespace arn
