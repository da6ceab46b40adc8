// ar_block_rmsnorm and ar_block_rmsnorm_i8: checks, launch shape, launch.
#include "block_norm.cuh"

namespace arn {

// Rows above 8 * 8192 columns need clusters of 16 CTAs, beyond the portable
// size: allowed by each call that needs them (a host-side attribute).
static cudaError_t allow_wide_clusters(BlockNormKernel kern) {
  return cudaFuncSetAttribute(reinterpret_cast<const void *>(kern),
                              cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

// Packs of a thread where there are rows enough for a CTA each.  A norm after the
// block is a second sum that a row has to wait for: four packs a thread, half as
// many warps to meet and more loads under way in each (8192 rows of 6144, one
// partial: 61.4 us, with two packs 79 us).  Without it, and with so many
// partials that loads are under way anyway, two packs keep more threads (4096
// rows of 8192: four partials and the norm 69 us against 74 us, two without it
// 59 us against 66 us).
static int packs_a_thread(int n, bool post) { return post && n <= 3 ? 4 : 2; }

static int run_block_norm(const void *const *partials, int n, int type, const void *post_weight,
                          const void *gate, int64_t gate_stride, int64_t gate_rows,
                          float block_scale, const void *residual, int residual_type,
                          float residual_scale, const void *weight, float weight_offset, float eps,
                          int64_t m, int64_t H, void *out, float *scales, void *residual_out,
                          bool bytes, void *stream) {
  const int st0 = check_shape(n, m, H, eps);
  if (st0 != AR_OK) return st0;
  if (!is_16bit(type) || (residual_type != type && residual_type != AR_TYPE_F32)) return AR_ERR_ARG;
  if (!std::isfinite(block_scale) || !std::isfinite(residual_scale) || !std::isfinite(weight_offset))
    return AR_ERR_ARG;
  const int64_t gates = gate != nullptr && m > 0 && gate_rows > 0 ? (m - 1) / gate_rows + 1 : 0;
  if (gate != nullptr) {
    if (gate_rows < 1) return AR_ERR_ARG;
    if (gates > 1) {
      if (gate_stride < H) return AR_ERR_ARG;
      if (gate_stride % kPackElems != 0) return AR_ERR_ALIGN;
      if (gate_stride > (int64_t{1} << 40) / gates) return AR_ERR_UNSUPPORTED;
    }
  }
  if (m == 0) return AR_OK;
  if (!partials || !residual || !weight || !out || !residual_out || (bytes && !scales))
    return AR_ERR_ARG;
  for (int k = 0; k < n; ++k) {
    if (!partials[k]) return AR_ERR_ARG;
  }
  for (int k = 0; k < n; ++k) {
    if (!aligned16(partials[k])) return AR_ERR_ALIGN;
  }
  if (!aligned16(post_weight) || !aligned16(gate) || !aligned16(residual) || !aligned16(weight) ||
      !aligned16(out) || !aligned16(residual_out) || !aligned_to(scales, 4))
    return AR_ERR_ALIGN;
  const int64_t rsize = type_size(residual_type), row2 = H * 2;
  const Range o = range_of(out, m * H * (bytes ? 1 : 2)), ro = range_of(residual_out, m * H * rsize);
  const Range sc = range_of(scales, bytes ? m * 4 : 0);
  const Range in[4] = {range_of(post_weight, post_weight ? row2 : 0),
                       range_of(gate, gates > 0 ? ((gates - 1) * gate_stride + H) * 2 : 0),
                       range_of(weight, row2), range_of(residual, m * H * rsize)};
  for (int i = 0; i < 4; ++i) {
    if (overlap(o, in[i]) || overlap(sc, in[i])) return AR_ERR_ALIAS;
    if (overlap(ro, in[i]) && !(i == 3 && residual_out == residual)) return AR_ERR_ALIAS;
  }
  for (int k = 0; k < n; ++k) {
    const Range p = range_of(partials[k], m * row2);
    if (overlap(o, p) || overlap(ro, p) || overlap(sc, p)) return AR_ERR_ALIAS;
  }
  if (overlap(o, ro) || overlap(o, sc) || overlap(ro, sc)) return AR_ERR_ALIAS;
  int st;
  DeviceState *d = current_device(&st);
  if (!d) return st;
  BlockNormArgs a = {};
  for (int k = 0; k < n; ++k) a.p[k] = static_cast<const uint4 *>(partials[k]);
  a.post = static_cast<const uint4 *>(post_weight);
  a.gate = static_cast<const uint4 *>(gate);
  a.res = static_cast<const uint4 *>(residual);
  a.w = static_cast<const uint4 *>(weight);
  a.out = out;
  a.scales = bytes ? scales : nullptr;
  a.rout = static_cast<uint4 *>(residual_out);
  a.m = m;
  a.gate_stride = gate_stride / kPackElems;
  a.gate_rows = gate != nullptr ? gate_rows : 1;
  a.n = n;
  a.P = static_cast<int>(H / kPackElems);
  a.H = static_cast<float>(H);
  a.eps = eps;
  a.block_scale = block_scale;
  a.residual_scale = residual_scale;
  a.offset = weight_offset;
  a.wait_limit_ns = kWaitLimitNs;
  a.status = d->status;
  // CTAs a row: as many as leave each 64 packs while the grid is below one
  // CTA an SM, up to 8; at least as many as hold the row in registers.
  int S = 1, vpt = 1;
  while (S < 8 && m * S * 2 <= d->sms && a.P / (S * 2) >= 64) S *= 2;
  const bool few = S > 1;
  while ((a.P + S - 1) / S > kMaxPacksPerCta) S *= 2;
  if (!few) vpt = S > 1 ? 4 : packs_a_thread(n, post_weight != nullptr);
  a.per_cta = (a.P + S - 1) / S;
  a.split = S;
  const int threads = ((a.per_cta + vpt - 1) / vpt + 31) / 32 * 32;
  if (m > INT32_MAX / S) return AR_ERR_UNSUPPORTED;
  int registers;
  const bool r32 = residual_type == AR_TYPE_F32;
  const BlockNormKernel kern = type == AR_TYPE_BF16 ? block_norm_bf16(r32, S > 1, vpt, &registers)
                                                    : block_norm_f16(r32, S > 1, vpt, &registers);
  if (S > 8 && allow_wide_clusters(kern) != cudaSuccess) {
    cudaGetLastError();
    return AR_ERR_CUDA;
  }
  if (!few) {  // a wave of CTAs, but not more rows than 26 MB of L2
    const int by_threads = 2048 / threads, by_registers = 65536 / (registers * threads);
    const int ctas = by_threads < by_registers ? by_threads : by_registers;
    const int64_t wave = static_cast<int64_t>(d->sms) * (ctas > 32 ? 32 : ctas) / S;
    const int64_t most = (int64_t{26} << 20) / (H * (2 * n + rsize));
    a.ahead = wave < most ? wave : most;
  }
  return launch_pdl(kern, a, m * S, threads, 0, S, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? AR_OK
             : AR_ERR_CUDA;
}

}  // namespace arn

using namespace arn;

extern "C" {

int ar_block_rmsnorm(const void *const *partials, int n, int type, const void *post_weight,
                     const void *gate, int64_t gate_stride, int64_t gate_rows, float block_scale,
                     const void *residual, int residual_type, float residual_scale,
                     const void *weight, float weight_offset, float eps, int64_t m, int64_t H,
                     void *out, void *residual_out, void *stream) {
  return run_block_norm(partials, n, type, post_weight, gate, gate_stride, gate_rows, block_scale,
                        residual, residual_type, residual_scale, weight, weight_offset, eps, m, H,
                        out, nullptr, residual_out, false, stream);
}

int ar_block_rmsnorm_i8(const void *const *partials, int n, int type, const void *post_weight,
                        const void *gate, int64_t gate_stride, int64_t gate_rows,
                        float block_scale, const void *residual, int residual_type,
                        float residual_scale, const void *weight, float weight_offset, float eps,
                        int64_t m, int64_t H, int8_t *q, float *scales, void *residual_out,
                        void *stream) {
  return run_block_norm(partials, n, type, post_weight, gate, gate_stride, gate_rows, block_scale,
                        residual, residual_type, residual_scale, weight, weight_offset, eps, m, H, q,
                        scales, residual_out, true, stream);
}

}  // extern "C"
