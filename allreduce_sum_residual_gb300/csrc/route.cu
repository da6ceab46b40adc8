// Routing to experts (ar_route_experts): scores, groups, top-k, weights.
//
// One warp takes one token.  A group of experts lies on L = 32 / 2^ceil(log2
// groups) neighbouring lanes, V = ceil(group size / L) neighbouring experts
// on each, so that (lane, register) order is expert order: "lowest index of
// the largest" is the lowest lane of a ballot, then its lowest register.
// A group's score is a butterfly over its L lanes.  The k rounds of the
// top-k are one integer max over the warp (redux) and one ballot each, on
// keys that order like the choices.
//
// Equal to 64 bits.  A choice computed in fp32 is off by a few 2^-24, so two
// experts that close can come out in the wrong order, and with 256 experts
// that happens about once in a thousand rows.  The kernel therefore also
// finds the (k+1)-th choice, and a row in which two neighbours of that order
// (or the last kept and the first dropped group) are nearer than the error
// bound is done again in fp64 by its warp.  Neighbours with the same logit
// and bias are exact ties, which need no second look, and so does nothing
// where the choices rank as the logits: those are compared as they are.
#include <cuda_fp16.h>

#include <cmath>
#include <type_traits>

#include "experts.cuh"

namespace arn {

struct RouteArgs {
  const void *x;
  const float *bias;
  float *w;
  int32_t *ids;
  int64_t m, stride;
  int E, k;
  int groups, topk_groups, gs;  // gs: experts per group
  int lanes_log2;               // lanes per group
  int softmax, top2, renorm;
  int by_logit;  // choices rank as the logits: no bias, groups by their maximum
  int vec;       // every lane's V logits are one aligned vector inside its group
  float scale;
  int *status;
};

constexpr int kRouteWarps = 4;

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }

// Signed keys that order as the numbers do.  kOut: not a candidate (taken,
// or in a dropped group); kOut + 1: an expert that is off.  Every number
// above -inf has a larger key than both.
__device__ __forceinline__ int order_key(float c) {
  const int b = __float_as_int(c + 0.f);  // -0 becomes +0: they are equal
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ long long order_key(double c) {
  const long long b = __double_as_longlong(c + 0.0);
  return b ^ ((b >> 63) & 0x7FFFFFFFFFFFFFFFll);
}
template <typename F>
struct Key;
template <>
struct Key<float> {
  using type = int;
  static constexpr int kOut = INT32_MIN;
};
template <>
struct Key<double> {
  using type = long long;
  static constexpr long long kOut = INT64_MIN;
};

__device__ __forceinline__ int warp_max(int v) { return __reduce_max_sync(0xFFFFFFFFu, v); }
__device__ __forceinline__ long long warp_max(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const long long u = __shfl_xor_sync(0xFFFFFFFFu, v, o);
    v = u > v ? u : v;
  }
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
template <typename F>
__device__ __forceinline__ F warp_total(F v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ float exponential(float v) { return expf(v); }
__device__ __forceinline__ double exponential(double v) { return exp(v); }

// The softmax maximum and sum of a row, enough to compute any score again.
template <typename F>
struct Scale {
  F top, sum;
};

template <typename F, int V>
__device__ __forceinline__ Scale<F> scale_of(const float (&x)[V]) {
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) top = fmaxf(top, x[i]);
  top = warp_max(top);
  Scale<F> s;
  s.top = top > -INFINITY ? F(top) : F(0);  // nothing on: every exp is 0
  F sum = F(0);
#pragma unroll
  for (int i = 0; i < V; ++i) sum += exponential(F(x[i]) - s.top);
  s.sum = warp_total(sum);
  return s;
}

template <typename F>
__device__ __forceinline__ F score_of(const RouteArgs &a, F x, const Scale<F> &s) {
  if (a.softmax) return exponential(x - s.top) / s.sum;
  return F(1) / (F(1) + exponential(-x));
}

// The choice of an expert that is on; -inf otherwise (off, or NaN).
template <typename F>
__device__ __forceinline__ F choice_of(const RouteArgs &a, float x, float bias, const Scale<F> &s) {
  if (!(x > -INFINITY)) return F(-INFINITY);
  const F c = a.by_logit ? F(x) : score_of<F>(a, F(x), s) + F(bias);
  return c > F(-INFINITY) ? c : F(-INFINITY);
}

// The order of a row: lane j <= k returns the id of its (j+1)-th choice (-1
// where there are fewer candidates).  *close: whether the group border is
// nearer than the error of two group scores, 2 delta; the caller looks at
// the rest.  x: this lane's logits, of which those in `valid` exist.
template <typename F, int V>
__device__ __forceinline__ int order_row(const RouteArgs &a, const float (&x)[V], uint32_t valid,
                                         int first, const Scale<F> &sc, F delta, bool *close) {
  using K = typename Key<F>::type;
  constexpr K kOut = Key<F>::kOut, kDead = kOut + 1;
  const int lane = threadIdx.x & 31;
  K key[V];
  F hi = F(-INFINITY), second = F(-INFINITY);  // this lane's two largest choices
#pragma unroll
  for (int i = 0; i < V; ++i) {
    key[i] = kOut;
    if (valid >> i & 1u) {
      const float b = a.bias != nullptr ? __ldg(a.bias + first + i) : 0.f;
      const F c = choice_of<F>(a, x[i], b, sc);
      key[i] = c > F(-INFINITY) ? order_key(c) : kDead;
      if (c > hi) {
        second = hi;
        hi = c;
      } else if (c > second) {
        second = c;
      }
    }
  }
  *close = false;
  if (a.topk_groups < a.groups) {
    for (int o = 1; o < 1 << a.lanes_log2; o <<= 1) {
      const F h = __shfl_xor_sync(0xFFFFFFFFu, hi, o), s = __shfl_xor_sync(0xFFFFFFFFu, second, o);
      second = hi > h ? (second > h ? second : h) : (hi > s ? hi : s);
      hi = hi > h ? hi : h;
    }
    // -inf with too few experts that are on
    const F mine = !a.top2 ? hi : second > F(-INFINITY) ? hi + second : F(-INFINITY);
    const int group = lane >> a.lanes_log2;
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const F other = __shfl_sync(0xFFFFFFFFu, mine, g << a.lanes_log2);
      rank += g != group && (other > mine || (other == mine && g < group)) ? 1 : 0;
    }
    const bool kept = rank < a.topk_groups;
    F above = F(INFINITY), below = F(-INFINITY);  // border: the worst kept, the best dropped
    for (int g = 0; g < a.groups; ++g) {
      const F other = __shfl_sync(0xFFFFFFFFu, mine, g << a.lanes_log2);
      const bool in = __shfl_sync(0xFFFFFFFFu, kept ? 1 : 0, g << a.lanes_log2) != 0;
      if (in) above = other < above ? other : above;
      else below = other > below ? other : below;
    }
    // Dropped groups at -inf are below every number, and -inf equals -inf.
    *close = below > F(-INFINITY) && !(above - below > delta + delta);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (!kept) key[i] = kOut;
  }
  K best = kOut;
#pragma unroll
  for (int i = 0; i < V; ++i) best = key[i] > best ? key[i] : best;
  int id = -1;
  for (int r = 0; r <= a.k; ++r) {
    const K top = warp_max(best);
    if (top == kOut) break;  // the same in every lane
    const int src = __ffs(__ballot_sync(0xFFFFFFFFu, best == top)) - 1;
    int at = -1;
    K next = kOut;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool it = lane == src && at < 0 && key[i] == top;
      if (it) {
        at = first + i;
        key[i] = kOut;
      }
      next = key[i] > next ? key[i] : next;
    }
    best = next;
    at = __shfl_sync(0xFFFFFFFFu, at, src);
    if (lane == r) id = at;
  }
  return id;
}

// The same row in fp64, out of the way of the common path's registers.
template <int V>
__device__ __noinline__ int order_row_64(const RouteArgs &a, const float (&x)[V], uint32_t valid,
                                         int first) {
  bool close;
  Scale<double> s{0.0, 1.0};
  if (a.softmax) s = scale_of<double, V>(x);
  return order_row<double, V>(a, x, valid, first, s, 0.0, &close);
}

template <typename T, int V>
__global__ void __launch_bounds__(kRouteWarps * 32) k_route(const __grid_constant__ RouteArgs a) {
  const int lane = threadIdx.x & 31;
  const int group = lane >> a.lanes_log2;
  const int in_group = (lane & ((1 << a.lanes_log2) - 1)) * V;
  const int first = group * a.gs + in_group;  // this lane's first expert
  int count = group < a.groups ? a.gs - in_group : 0;
  count = count < 0 ? 0 : count < V ? count : V;
  // Checking build: the lane's experts exist.
  if (!in_bounds(count == 0 || (first >= 0 && first + count <= a.E), a.status)) count = 0;
  const uint32_t valid = count >= 32 ? 0xFFFFFFFFu : (1u << count) - 1u;
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5); row < a.m;
       row += static_cast<int64_t>(gridDim.x) * kRouteWarps) {
    const T *p = static_cast<const T *>(a.x) + row * a.stride;
    float x[V];
    if (a.vec) {
      constexpr int kBytes = V * static_cast<int>(sizeof(T));
      using W = typename std::conditional<
          kBytes % 16 == 0, uint4,
          typename std::conditional<
              kBytes % 8 == 0, uint2,
              typename std::conditional<kBytes % 4 == 0, uint32_t, uint16_t>::type>::type>::type;
      constexpr int kWords = kBytes / static_cast<int>(sizeof(W));
      W w[kWords];
      T t[V];
      static_assert(sizeof(w) == sizeof(t), "one vector is V logits");
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        if (count > 0) w[i] = __ldg(reinterpret_cast<const W *>(p + first) + i);
      memcpy(t, w, sizeof t);
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = count > 0 ? to_float(t[i]) : -INFINITY;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = i < count ? to_float(p[first + i]) : -INFINITY;
    }
    // Softmax needs the row's sum only for scores: not for choices that rank
    // as the logits, nor for weights that are renormalised.
    Scale<float> sc{0.f, 1.f};
    if (a.softmax && !(a.by_logit && a.renorm)) sc = scale_of<float, V>(x);
    // Error bound of the difference of two fp32 choices, in 2^-24 of the
    // largest choice.  A sigmoid (exp within 1 ulp, an add, a divide) is off
    // by 4, a softmax score by 4 and its row's sum of up to 37 rounded adds,
    // the sum with the bias by 1; twice that is under 2^-20 and 2^-17.
    float delta = 0.f;
    if (!a.by_logit) {
      float big = 1.f;
      if (a.bias != nullptr) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i < count) {
            const float b = fabsf(__ldg(a.bias + first + i));
            if (b < INFINITY) big = fmaxf(big, 1.f + b);  // an infinite choice is exact
          }
        big = warp_max(big);
      }
      delta = big * (a.softmax ? 0x1p-17f : 0x1p-20f);
    }
    bool close;
    int id = order_row<float, V>(a, x, valid, first, sc, delta, &close);
    float xs = id >= 0 ? to_float(p[id]) : -INFINITY;
    if (!a.by_logit) {
      const float bs = id >= 0 && a.bias != nullptr ? __ldg(a.bias + id) : 0.f;
      const float c = id >= 0 ? choice_of<float>(a, xs, bs, sc) : -INFINITY;
      const float cn = __shfl_down_sync(0xFFFFFFFFu, c, 1);
      const float xn = __shfl_down_sync(0xFFFFFFFFu, xs, 1);
      const float bn = __shfl_down_sync(0xFFFFFFFFu, bs, 1);
      const bool near = lane < a.k && cn > -INFINITY && !(c - cn > delta) &&
                        !(xs == xn && bs == bn);
      if (__any_sync(0xFFFFFFFFu, near || close)) {
        id = order_row_64<V>(a, x, valid, first);
        xs = id >= 0 ? to_float(p[id]) : -INFINITY;
      }
    }
    float w = 0.f;
    if (a.softmax && a.renorm) {
      // Relative to the largest chosen logit: the row's sum cancels, and the
      // chosen cannot all underflow.
      const float t = warp_max(lane < a.k ? xs : -INFINITY);
      if (lane < a.k && t > -INFINITY) w = expf(xs - t);
      bool poison = false;  // a NaN or +inf anywhere in the row makes every score NaN
#pragma unroll
      for (int i = 0; i < V; ++i) poison |= i < count && !(x[i] < INFINITY);
      if (__any_sync(0xFFFFFFFFu, poison)) w = __int_as_float(0x7FC00000);
    } else if (lane < a.k) {
      w = sc.sum == 0.f ? 0.f : score_of<float>(a, xs, sc);  // 0: a row with nothing on
    }
    if (a.renorm) {
      const float total = warp_total(lane < a.k ? w : 0.f);
      w = total == 0.f ? 0.f : w / total;
    }
    if (lane < a.k) {
      a.w[row * a.k + lane] = w * a.scale;
      a.ids[row * a.k + lane] = id;
    }
  }
}

using RouteKernel = void (*)(RouteArgs);

template <typename T>
static RouteKernel route_kernel(int v) {
  switch (v) {
    case 1: return &k_route<T, 1>;
    case 2: return &k_route<T, 2>;
    case 4: return &k_route<T, 4>;
    case 8: return &k_route<T, 8>;
    case 16: return &k_route<T, 16>;
    default: return &k_route<T, 32>;
  }
}

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
  RouteKernel kern = logits_type == AR_TYPE_F32 ? route_kernel<float>(v)
                     : logits_type == AR_TYPE_BF16 ? route_kernel<__nv_bfloat16>(v)
                                                   : route_kernel<__half>(v);
  int64_t grid = (m + kRouteWarps - 1) / kRouteWarps;
  const int64_t cap = static_cast<int64_t>(d->sms) * 16;
  if (grid > cap) grid = cap;
  return launch_pdl(kern, a, grid, kRouteWarps * 32, 0, 1, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? AR_OK
             : AR_ERR_CUDA;
}
