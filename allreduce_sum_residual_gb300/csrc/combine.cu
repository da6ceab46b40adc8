// The weighted sum of each token's expert outputs (ar_combine), and the same
// sum through the residual add and RMSNorm (ar_combine_rmsnorm).
//
//   r[i, c] = shared[i, c] + sum_j w[i, j] y[slot[i, j], c]   (+ residual)
//
// Bound by memory: a row reads up to k + 2 rows and writes one or two, and
// the sum stays in registers until its row's square sum is known.  The split
// is the fused epilogue's: a CTA, or a cluster of them at few rows, takes
// one row, a thread one pack.  The k row numbers and weights of a token are
// read once per warp, one a lane, and broadcast by shuffles.
//
// What made it fast, at 8192 tokens of 8 choices and 6144 columns (1.1 GB,
// 163 us at the rate of a plain copy): 226 us with one 768-thread CTA an SM,
// whose loads, square sum and stores follow one another; 175 us with two,
// which takes at most 40 registers, hence four rows in flight and the
// residual and the gain loaded late; 161 us with the rows of the token one
// wave of CTAs ahead prefetched into L2 (their numbers are in slots).  The
// partial alone needs no CTA to hold a row: 256-thread CTAs, eight an SM (777
// tokens of 6 choices, half of them here, 7168 columns: 10.5 us, 16.4 us with
// a CTA a row).
#include "experts.cuh"

namespace arn {

struct CombineArgs {
  const uint4 *y;          // [rows, P] packs
  const int32_t *slots;    // [m, k], or null: row i * k + j
  const float *weights;    // [m, k]
  const uint4 *shared;     // [m, P], or null
  const uint4 *res;        // [m, P] (norm)
  const uint4 *w;          // [P] (norm)
  uint4 *out;
  uint4 *rout;             // (norm)
  int64_t m, rows;
  int k, P, per_cta;
  int split;               // CTAs of a row (norm: one cluster)
  int64_t ahead;           // rows to prefetch ahead (norm, one CTA a row); 0: none
  float H, eps;
  uint64_t wait_limit_ns;
  int *status;
};

// U: rows of y in flight at a time.  Threads of a CTA at most, CTAs of an SM
// at least (the register budget).
template <int U, int THREADS, int CTAS, bool NORM, bool CL>
__global__ void __launch_bounds__(THREADS, CTAS) k_combine(const __grid_constant__ CombineArgs a) {
  __shared__ float red[33];
  __shared__ float cta_totals[kMaxClusterCtas];
  __shared__ uint64_t totals_bar;
  __shared__ int totals_abort;

  const uint32_t S = static_cast<uint32_t>(a.split);
  const uint32_t q = CL ? cluster_ctarank() : blockIdx.x % S;
  const int64_t row = blockIdx.x / S;
  const int c0 = static_cast<int>(q) * a.per_cta;
  const int c1 = min(a.P, c0 + a.per_cta);
  const int64_t base = row * static_cast<int64_t>(a.P);
  const int T = blockDim.x;
  const int lane = threadIdx.x & 31;
  // Checking build: the row, its pack range, and threads for all of it.
  const bool live = in_bounds(row < a.m && c0 >= 0 && (c1 <= c0 || c1 - c0 <= T) &&
                                  a.k >= 1 && a.k <= AR_MAX_TOPK &&
                                  (!CL || S <= static_cast<uint32_t>(kMaxClusterCtas)) && q < S,
                              a.status);
  if constexpr (CL) {
    if (threadIdx.x == 0) {
      mbar_init(&totals_bar, 1);
      totals_abort = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    cluster_arrive_release();
  }
  pdl_wait_prior_grid();
  pdl_launch_dependents();

  // Lane j: the row of y and the weight of choice j; -1 for none.
  int64_t my_row = -1;
  float my_w = 0.f;
  if (live && lane < a.k) {
    const int64_t p = row * a.k + lane;
    my_row = a.slots != nullptr ? static_cast<int64_t>(__ldg(a.slots + p)) : p;
    if (my_row < 0 || my_row >= a.rows) my_row = -1;
    const float w = __ldg(a.weights + p);
    if (my_row >= 0) my_w = w;
  }
  const int c = c0 + static_cast<int>(threadIdx.x);
  const bool in = live && c < c1;
  // Clusters load the residual and the gain with the rows (fewer trips in a
  // row); one CTA a row loads them late (fewer registers, more CTAs an SM).
  uint4 rv = make_uint4(0, 0, 0, 0), wv = rv;
  if constexpr (NORM && CL) {
    if (in) {
      rv = ld_ro(a.res + base + c);
      wv = ld_ro(a.w + c);
    }
  }
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (in && a.shared != nullptr) unpack8(ld_ro(a.shared + base + c), acc);
  for (int j0 = 0; j0 < a.k; j0 += U) {
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // Lanes behind k hold no row: the shuffle gives -1 there.
      const int64_t at = __shfl_sync(0xFFFFFFFFu, my_row, (j0 + u) & 31);
      x[u] = make_uint4(0, 0, 0, 0);
      if (in && at >= 0) x[u] = ld_ro(a.y + at * a.P + c);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float wj = __shfl_sync(0xFFFFFFFFu, my_w, (j0 + u) & 31);
      float f[8];
      unpack8(x[u], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(wj, f[e], acc[e]);
    }
  }
  if constexpr (!NORM) {
    if (in) st_stream(a.out + base + c, pack8(acc));
    return;
  }
  if constexpr (!CL) {
    if (in) rv = ld_ro(a.res + base + c);
    // The rows of the token one wave of CTAs ahead, on their way to L2.
    if (live && a.ahead > 0 && row + a.ahead < a.m && threadIdx.x <= a.k) {
      const uint32_t bytes = static_cast<uint32_t>(a.P) * 16u;
      if (threadIdx.x == a.k) {
        prefetch_l2(a.res + base + a.ahead * a.P, bytes);
      } else {
        const int64_t p = (row + a.ahead) * a.k + threadIdx.x;
        const int64_t at = a.slots != nullptr ? static_cast<int64_t>(__ldg(a.slots + p)) : p;
        if (at >= 0 && at < a.rows) prefetch_l2(a.y + at * a.P, bytes);
      }
    }
  }
  float rs[8];
  unpack8(rv, rs);
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    acc[e] += rs[e];
    ss = fmaf(acc[e], acc[e], ss);
  }
  if (in) st_stream(a.rout + base + c, pack8(acc));
  if constexpr (!CL) {
    if (in) wv = ld_ro(a.w + c);
  }
  float total = block_sum(in ? ss : 0.f, red);
  if constexpr (CL) {
    // As in the fused epilogue: every CTA sends its total to every CTA of
    // the row, which adds them in rank order; a bounded wait.
    cluster_wait_acquire();
    if (threadIdx.x == 0)
      mbar_arrive_expect_tx(&totals_bar, S * static_cast<uint32_t>(sizeof(float)));
    if (threadIdx.x < S) st_async_remote_f32(&cta_totals[q], threadIdx.x, total, &totals_bar);
    mbar_wait_bounded(&totals_bar, 0, &totals_abort, a.wait_limit_ns, a.status);
    total = 0.f;
    for (uint32_t s = 0; s < S; ++s) total += cta_totals[s];
  }
  const float inv = rsqrtf(total / a.H + a.eps);
  if (in) {
    float w[8], o[8];
    unpack8(wv, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = (acc[e] * inv) * w[e];
    st_stream(a.out + base + c, pack8(o));
  }
}

using CombineKernel = void (*)(CombineArgs);

// Rows above 8 * 8192 columns need clusters of 16 CTAs, beyond the portable
// size: allowed by each call that needs them (a host-side attribute).
static cudaError_t allow_wide_clusters() {
  return cudaFuncSetAttribute(reinterpret_cast<const void *>(&k_combine<8, 1024, 1, true, true>),
                              cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

static int run_combine(const void *y, int64_t rows, const int32_t *slots, const float *weights,
                       const void *shared, const void *residual, const void *weight, float eps,
                       int64_t m, int k, int64_t H, void *out, void *residual_out, bool norm,
                       void *stream) {
  const int st0 = check_shape(1, m, H, eps);
  if (st0 != AR_OK) return st0;
  if (k < 1 || rows < 0) return AR_ERR_ARG;
  if (k > AR_MAX_TOPK) return AR_ERR_UNSUPPORTED;
  if (m > (int64_t{1} << 40) / (H * k) || rows > (int64_t{1} << 40) / H) return AR_ERR_UNSUPPORTED;
  if (slots == nullptr && rows != m * k) return AR_ERR_ARG;
  if (m == 0) return AR_OK;
  if ((!y && rows > 0) || !weights || !out || (norm && (!residual || !weight || !residual_out)))
    return AR_ERR_ARG;
  if (!aligned16(y) || !aligned16(shared) || !aligned16(out) || !aligned_to(slots, 4) ||
      !aligned_to(weights, 4) ||
      (norm && (!aligned16(residual) || !aligned16(weight) || !aligned16(residual_out))))
    return AR_ERR_ALIGN;
  const int64_t bytes = m * H * 2;
  const Range o = range_of(out, bytes), ro = range_of(residual_out, norm ? bytes : 0);
  const Range in[6] = {range_of(y, rows * H * 2), range_of(slots, slots ? m * k * 4 : 0),
                       range_of(weights, m * k * 4), range_of(shared, shared ? bytes : 0),
                       range_of(residual, norm ? bytes : 0), range_of(weight, norm ? H * 2 : 0)};
  for (int i = 0; i < 6; ++i) {
    if (overlap(o, in[i])) return AR_ERR_ALIAS;
    if (norm && overlap(ro, in[i]) && !(i == 4 && residual_out == residual)) return AR_ERR_ALIAS;
  }
  if (norm && overlap(o, ro)) return AR_ERR_ALIAS;
  int st;
  DeviceState *d = current_device(&st);
  if (!d) return st;
  CombineArgs a = {};
  a.y = static_cast<const uint4 *>(y);
  a.slots = slots;
  a.weights = weights;
  a.shared = static_cast<const uint4 *>(shared);
  a.res = static_cast<const uint4 *>(residual);
  a.w = static_cast<const uint4 *>(weight);
  a.out = static_cast<uint4 *>(out);
  a.rout = static_cast<uint4 *>(residual_out);
  a.m = m;
  a.rows = rows;
  a.k = k;
  a.P = static_cast<int>(H / kPackElems);
  a.H = static_cast<float>(H);
  a.eps = eps;
  a.wait_limit_ns = kWaitLimitNs;
  a.status = d->status;
  // With a norm: CTAs a row, as many as leave each 64 packs while the grid
  // is below one CTA an SM, up to 8; at least as many as hold the row in
  // registers.  Without one, the CTAs of a row share nothing and take 256
  // packs each.
  int S = 1;
  if (norm) {
    while (S < 8 && m * S * 2 <= d->sms && a.P / (S * 2) >= 64) S *= 2;
    while ((a.P + S - 1) / S > kMaxPacksPerCta) S *= 2;
  } else {
    S = (a.P + 255) / 256;
  }
  a.per_cta = (a.P + S - 1) / S;
  a.split = S;
  const int threads = (a.per_cta + 31) / 32 * 32;
  if (m > INT32_MAX / S) return AR_ERR_UNSUPPORTED;
  if (norm && S > 8 && allow_wide_clusters() != cudaSuccess) {
    cudaGetLastError();
    return AR_ERR_CUDA;
  }
  CombineKernel kern = &k_combine<2, 256, 8, false, false>;
  if (norm && S > 1) {
    kern = &k_combine<8, 1024, 1, true, true>;
  } else if (norm) {
    // CTAs of an SM by the threads a row needs, and the distance of the
    // prefetch: a wave of them (with more than 768 threads half of one: 4096
    // tokens of 7168 columns in 93.5 us against 97 us).
    const int waves = threads <= 512 ? 3 : threads <= 768 ? 2 : 1;
    kern = threads <= 512   ? &k_combine<4, 512, 3, true, false>
           : threads <= 768 ? &k_combine<4, 768, 2, true, false>
                            : &k_combine<2, 1024, 2, true, false>;
    a.ahead = static_cast<int64_t>(d->sms) * waves;
  }
  return launch_pdl(kern, a, m * S, threads, 0, norm ? S : 1, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? AR_OK
             : AR_ERR_CUDA;
}

}  // namespace arn

using namespace arn;

extern "C" {

int ar_combine(const void *y, int64_t rows, const int32_t *slots, const float *weights,
               const void *shared, int64_t m, int k, int64_t H, void *out, void *stream) {
  return run_combine(y, rows, slots, weights, shared, nullptr, nullptr, 0.f, m, k, H, out, nullptr,
                     false, stream);
}

int ar_combine_rmsnorm(const void *y, int64_t rows, const int32_t *slots, const float *weights,
                       const void *shared, const void *residual, const void *weight, float eps,
                       int64_t m, int k, int64_t H, void *out, void *residual_out, void *stream) {
  return run_combine(y, rows, slots, weights, shared, residual, weight, eps, m, k, H, out,
                     residual_out, true, stream);
}

}  // extern "C"
