// ar_route_experts: checks and the launch.  The kernels (route.cuh) are
// compiled in route_<logits' type>.cu.
#include "route.cuh"

namespace arn {

RouteKernel route_kernel_f32(int v, RouteBy by);
RouteKernel route_kernel_bf16(int v, RouteBy by);
RouteKernel route_kernel_f16(int v, RouteBy by);

}  // namespace arn

using namespace arn;

extern "C" int ar_route_experts(const void *logits, int logits_type, int64_t row_stride,
                                const float *bias, int64_t m, int E, int k, int scoring,
                                int groups, int topk_groups, int group_score, int renorm,
                                float scale, float *weights, int32_t *ids, void *stream) {
  const int size = type_size(logits_type);
  if (size == 0 || m < 0 || E < 1 || k < 1 || groups < 1 || groups > 32 || topk_groups < 1 ||
      topk_groups > groups)
    return AR_ERR_ARG;
  if (E > AR_MAX_EXPERTS || k > AR_MAX_TOPK) return AR_ERR_UNSUPPORTED;
  if (E % groups != 0) return AR_ERR_ARG;
  const int gs = E / groups;
  if (k > topk_groups * gs || row_stride < E || !std::isfinite(scale) ||
      (scoring != AR_SCORE_SOFTMAX && scoring != AR_SCORE_SIGMOID) ||
      (group_score != AR_GROUP_MAX && group_score != AR_GROUP_TOP2) ||
      (renorm != 0 && renorm != 1) || (groups > 1 && group_score == AR_GROUP_TOP2 && gs < 2))
    return AR_ERR_ARG;
  if (m > (int64_t{1} << 40) / row_stride || m > (int64_t{1} << 40) / k) return AR_ERR_UNSUPPORTED;
  if (m == 0) return AR_OK;
  if (!logits || !weights || !ids) return AR_ERR_ARG;
  if (!aligned_to(logits, size) || !aligned_to(bias, 4) || !aligned_to(weights, 4) ||
      !aligned_to(ids, 4))
    return AR_ERR_ALIGN;
  const Range wr = range_of(weights, m * k * 4), ir = range_of(ids, m * k * 4);
  const Range xr = range_of(logits, ((m - 1) * row_stride + E) * size);
  if (overlap(wr, ir) || overlap(wr, xr) || overlap(ir, xr)) return AR_ERR_ALIAS;
  if (bias != nullptr) {
    const Range br = range_of(bias, E * 4);
    if (overlap(wr, br) || overlap(ir, br)) return AR_ERR_ALIAS;
  }
  int st;
  DeviceState *d = current_device(&st);
  if (!d) return st;
  RouteArgs a = {};
  a.x = logits;
  a.bias = bias;
  a.w = weights;
  a.ids = ids;
  a.m = m;
  a.stride = row_stride;
  a.E = E;
  a.k = k;
  a.groups = groups;
  a.topk_groups = topk_groups;
  a.gs = gs;
  int gp_log2 = 0;
  while ((1 << gp_log2) < groups) ++gp_log2;
  a.lanes_log2 = 5 - gp_log2;
  const int lanes = 1 << a.lanes_log2;
  int v = 1;
  while (v * lanes < gs) v *= 2;  // at most 32: 2^ceil(log2 groups) < 2 groups
  a.softmax = scoring == AR_SCORE_SOFTMAX;
  a.top2 = group_score == AR_GROUP_TOP2;
  a.renorm = renorm;
  a.by_logit = bias == nullptr && (!a.top2 || topk_groups == groups);
  const int vector = v * size % 16 == 0 ? 16 : v * size % 16;  // 2, 4, 8 or 16
  a.vec = gs % v == 0 && row_stride * size % vector == 0 && aligned_to(logits, vector);
  a.scale = scale;
  a.status = d->status;
  const RouteBy by = a.by_logit ? kByLogit : a.softmax ? kBySoftmax : kBySigmoid;
  RouteKernel kern = logits_type == AR_TYPE_F32    ? route_kernel_f32(v, by)
                     : logits_type == AR_TYPE_BF16 ? route_kernel_bf16(v, by)
                                                   : route_kernel_f16(v, by);
  int64_t grid = (m + kRouteWarps - 1) / kRouteWarps;
  const int64_t cap = static_cast<int64_t>(d->sms) * route_ctas(v);  // the bias is read once a warp
  if (grid > cap) grid = cap;
  return launch_pdl(kern, a, grid, kRouteWarps * 32, 0, 1, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? AR_OK
             : AR_ERR_CUDA;
}
