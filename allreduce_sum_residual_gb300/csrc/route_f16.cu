// Routing kernels for f16 logits.
#include "route.cuh"

namespace arn {

RouteKernel route_kernel_f16(int v, RouteBy by) { return route_kernel<__half>(v, by); }

}  // namespace arn
