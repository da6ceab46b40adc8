// Routing kernels for bf16 logits.
#include "route.cuh"

namespace arn {

RouteKernel route_kernel_bf16(int v, RouteBy by) { return route_kernel<__nv_bfloat16>(v, by); }

}  // namespace arn
