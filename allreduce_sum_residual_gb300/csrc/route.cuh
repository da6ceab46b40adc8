// Routing to experts (ar_route_experts): scores, groups, top-k, weights: the
// kernel.
//
// One warp takes one token.  A group of experts lies on L = 32 / 2^ceil(log2
// groups) neighbouring lanes, V = ceil(group size / L) neighbouring experts
// on each.  A group's score is a butterfly over its L lanes.
//
// Top-k.  Every choice becomes a 32-bit key, its order in the upper 23 bits
// and 511 - expert in the lower nine, so that keys are distinct and equal
// choices order by index.  A lane sorts its V keys (a merge network of max
// and min); a round is then one integer max over the warp (redux), which
// names the expert, and the lane that held it moves up its next key.
//
// Equal to 64 bits.  23 bits, and fp32 scores off by a few 2^-24, can put two
// experts in the wrong order.  The kernel therefore also finds the (k+1)-th
// choice and looks at neighbours of that order that are nearer than the error
// bound.  Where they are all that is near (a few rows in a thousand), the k +
// 1 sigmoids are computed again in fp64, one a lane, and sorted by those;
// otherwise (another expert near the last choice, or equal to it where one
// of these may have to make way; a group border too near to call; softmax
// scores) the warp does the whole row again, in fp64, or in fp32 where the
// choices rank as the logits and those are compared as they are.  Neighbours
// with the same logit and bias are exact ties, which need no second look.
//
// Bound by instructions, some 700 a row of 256 experts: 16384 such rows with
// groups and bias take 16.5 us (52 us with k passes over every lane's choices
// in place of the keys), where their bytes would take 2.6 us.
#pragma once

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
__device__ __forceinline__ F score_of(bool softmax, F x, const Scale<F> &s) {
  if (softmax) return exponential(x - s.top) / s.sum;
  return F(1) / (F(1) + exponential(-x));
}

// The choice of an expert that is on; -inf otherwise (off, or NaN).
template <typename F>
__device__ __forceinline__ F choice_of(const RouteArgs &a, float x, float bias, const Scale<F> &s) {
  if (!(x > -INFINITY)) return F(-INFINITY);
  const F c = a.by_logit ? F(x) : score_of<F>(a.softmax, F(x), s) + F(bias);
  return c > F(-INFINITY) ? c : F(-INFINITY);
}

// The order of a row, choice by choice in F: lane j <= k returns the id of its
// (j+1)-th choice (-1 where there are fewer candidates).  x: this lane's
// logits, of which those in `valid` exist.
template <typename F, int V>
__device__ __forceinline__ int order_row(const RouteArgs &a, const float (&x)[V], uint32_t valid,
                                         int first, const Scale<F> &sc) {
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

// Out of the way of the common path's registers.
template <int V>
__device__ __noinline__ int order_row_exactly(const RouteArgs &a, const float (&x)[V],
                                              uint32_t valid, int first) {
  if (a.by_logit) return order_row<float, V>(a, x, valid, first, Scale<float>{0.f, 1.f});
  Scale<double> s{0.0, 1.0};
  if (a.softmax) s = scale_of<double, V>(x);
  return order_row<double, V>(a, x, valid, first, s);
}

// Weights of a row with a chosen sigmoid score below e^-80, near fp32's end,
// where its share of the sum may still be any number: in fp64 up to the one
// rounding.
static __device__ __noinline__ float far_sigmoid_weight(float x, bool chosen, bool renorm, float scale) {
  double s = chosen ? score_of<double>(false, x, Scale<double>{0.0, 1.0}) : 0.0;
  if (renorm) {
    const double total = warp_total(s);
    s = total == 0.0 ? 0.0 : s / total;
  }
  return static_cast<float>(s * scale);
}

// A score to a few 2^-24 of 1, in few instructions: ex2.approx is off by 2
// ulp and its argument by half of one (of x - top or x, whose exponential or
// derivative makes up for its size), rcp.approx by 1; what they flush to zero
// is below 2^-126.
__device__ __forceinline__ float quick_exp2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float quick_inverse(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float quick_score(bool softmax, float x, float top, float inv) {
  constexpr float kLog2E = 1.44269504f;
  if (softmax) return quick_exp2((x - top) * kLog2E) * inv;
  return quick_inverse(1.f + quick_exp2(x * -kLog2E));
}

// A logit's order in the upper 23 bits, 2 or more; whole if it has 16.
template <bool EXACT>
__device__ __forceinline__ uint32_t logit_order(float x) {
  const uint32_t order = static_cast<uint32_t>(order_key(x)) ^ 0x80000000u;
  return (EXACT ? order >> 4 : order) & ~511u;  // a half widens to 19 bits
}

// Sorts descending (Batcher's odd-even merges; V a power of two).
template <int V>
__device__ __forceinline__ void sort_keys(uint32_t (&k)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int d = p; d >= 1; d /= 2)
#pragma unroll
      for (int j = d % p; j + d < V; j += 2 * d)
#pragma unroll
        for (int i = 0; i < d; ++i)
          if (i + j + d < V && (i + j) / (2 * p) == (i + j + d) / (2 * p)) {
            const uint32_t lo = min(k[i + j], k[i + j + d]), hi = max(k[i + j], k[i + j + d]);
            k[i + j] = hi;
            k[i + j + d] = lo;
          }
}

// CTAs an SM, by the registers: with six (80) the 16384 rows above take 16.5
// us, with eight (64), where more than the second look spills, 17.5 us, with
// five (96) 17.0 us.
constexpr int route_ctas(int v) { return v <= 8 ? 6 : v == 16 ? 4 : 2; }

// How experts are ordered: by their logits (a.by_logit), or by their scores
// with the bias.  The kind of score as a constant took 2.2 us off.
enum RouteBy { kByLogit, kBySigmoid, kBySoftmax };

template <typename T, int V, RouteBy BY>
__global__ void __launch_bounds__(kRouteWarps * 32, route_ctas(V))
    k_route(const __grid_constant__ RouteArgs a) {
  constexpr bool LOGIT = BY == kByLogit;
  const bool softmax = LOGIT ? a.softmax != 0 : BY == kBySoftmax;
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
  // The bias, and the range [-reach, 1 + reach] of the finite choices.
  float bias[V], reach = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    bias[i] = a.bias != nullptr && i < count ? __ldg(a.bias + first + i) : 0.f;
    const float b = fabsf(bias[i]);
    if (b < INFINITY) reach = fmaxf(reach, b);  // an infinite choice is exact
  }
  if (a.bias != nullptr) reach = warp_max(reach);
  // Keys in fixed point: `fine` steps in 1, from 3 (for -reach) on.  Adding
  // 2^23 leaves the rounded steps in an fp32's lower 23 bits.
  const float fine = 8388500.f / (1.f + 2.f * reach), base = fmaf(reach, fine, 3.f + 8388608.f);
  // How near two fp32 choices can be to come out in the wrong order.  In
  // 2^-24 of 1 + reach: a quick sigmoid is off by 6 at most, a softmax score
  // by 6 and its row's sum of up to 37 rounded adds, the sum with the bias by
  // 1, the key by 1.5 steps of 4: twice that is under 2^-19 and 2^-16.
  const float delta = (1.f + reach) * (softmax ? 0x1p-16f : 0x1p-19f);
  constexpr bool kExact = sizeof(T) == 2;  // keys that hold a logit whole
  constexpr uint32_t kTop = 8388600u;

  const int64_t step = static_cast<int64_t>(gridDim.x) * kRouteWarps;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5); row < a.m;
       row += step) {
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
    float inv = 1.f;
    if (softmax && !(LOGIT && a.renorm)) {
      sc = scale_of<float, V>(x);
      inv = 1.f / sc.sum;
    }
    // Keys.  0: no candidate; 1 in the upper bits: off; from 2 on the
    // choices, as fixed point (kTop: infinite), or the logits' own order.
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      uint32_t order;  // in the upper bits
      bool on = x[i] > -INFINITY;
      if constexpr (LOGIT) {
        order = logit_order<kExact>(x[i]);
      } else {
        const float c = quick_score(softmax, x[i], sc.top, inv) + bias[i];
        on = on && c > -INFINITY;
        order = __float_as_uint(fminf(fmaf(c, fine, base), 8388608.f + kTop)) << 9;
      }
      if (!on) order = 1u << 9;
      key[i] = i < count ? order + static_cast<uint32_t>(511 - first - i) : 0u;
    }
    sort_keys<V>(key);
    bool close = false;
    bool kept = true;
    if (a.topk_groups < a.groups) {
      uint32_t k1 = key[0], k2 = V > 1 ? key[1] : 0u;  // the group's two largest keys
      for (int o = 1; o < 1 << a.lanes_log2; o <<= 1) {
        const uint32_t q1 = __shfl_xor_sync(0xFFFFFFFFu, k1, o);
        const uint32_t q2 = __shfl_xor_sync(0xFFFFFFFFu, k2, o);
        k2 = max(min(k1, q1), max(k2, q2));
        k1 = max(k1, q1);
      }
      // Twice the group's score in the keys' steps; 2 with too few experts
      // that are on, 2 kTop with an infinite one.
      const uint32_t o1 = k1 >> 9, o2 = a.top2 ? k2 >> 9 : o1;
      uint32_t twice = o1 + (o1 == kTop ? o1 : o2);
      if (min(o1, o2) <= 1u) twice = 2u;
      // The groups' keys, and as many rounds as groups are kept.
      uint32_t score = group < a.groups ? (twice >> 1) << 9 | static_cast<uint32_t>(511 - group) : 0u;
      kept = false;
      uint32_t best = 0u;
      for (int r = 0; r < a.topk_groups; ++r) {
        best = __reduce_max_sync(0xFFFFFFFFu, score);
        if (score == best) {
          kept = true;
          score = 0u;
        }
      }
      kept = kept && group < a.groups;
      // The border: the worst kept, the best dropped.  Dropped groups at -inf
      // are below every number, and -inf equals -inf.
      const uint32_t next = __reduce_max_sync(0xFFFFFFFFu, score);
      if (next >> 9 > 1u) {
        if constexpr (LOGIT) {
          close = !kExact && best >> 9 == next >> 9;
        } else {
          const int last_lane = (511 - static_cast<int>(best & 511u)) << a.lanes_log2;
          const int next_lane = (511 - static_cast<int>(next & 511u)) << a.lanes_log2;
          const uint32_t above = __shfl_sync(0xFFFFFFFFu, twice, last_lane);
          const uint32_t below = __shfl_sync(0xFFFFFFFFu, twice, next_lane);
          // 2 steps for the halves that the keys leave out, 2 to be over
          // the line.
          close = static_cast<float>(static_cast<int>(above - below)) <= 2.f * delta * fine + 4.f;
        }
      }
      if (!LOGIT && close && !softmax) {  // the same in every lane
        // The border again in fp64: the groups' three largest keys, and the
        // two of group j computed by lane j.
        uint32_t k1 = key[0], k2 = V > 1 ? key[1] : 0u, k3 = V > 2 ? key[2] : 0u;
        for (int o = 1; o < 1 << a.lanes_log2; o <<= 1) {
          const uint32_t q1 = __shfl_xor_sync(0xFFFFFFFFu, k1, o);
          const uint32_t q2 = __shfl_xor_sync(0xFFFFFFFFu, k2, o);
          const uint32_t q3 = __shfl_xor_sync(0xFFFFFFFFu, k3, o);
          const uint32_t lo = min(k1, q1), hi2 = max(k2, q2);  // k1 >= k2 >= k3, the same for q
          k3 = max(max(k3, q3), min(lo, hi2));
          k3 = max(k3, min(k2, q2));
          k2 = max(lo, hi2);
          k1 = max(k1, q1);
        }
        const int leader = lane < a.groups ? lane << a.lanes_log2 : 0;
        const uint32_t g1 = __shfl_sync(0xFFFFFFFFu, k1, leader);
        const uint32_t g2 = __shfl_sync(0xFFFFFFFFu, k2, leader);
        const uint32_t g3 = __shfl_sync(0xFFFFFFFFu, k3, leader);
        auto exactly = [&](uint32_t of) -> double {
          if (of >> 9 <= 1u) return -INFINITY;
          const int e = 511 - static_cast<int>(of & 511u);
          return score_of<double>(softmax, to_float(p[e]), Scale<double>{0.0, 1.0}) +
                 (a.bias != nullptr ? __ldg(a.bias + e) : 0.f);
        };
        double sum = exactly(g1);
        if (a.top2) sum += exactly(g2);  // -inf with too few experts that are on
        // Whether the next in the group could be one of these after all.
        const uint32_t in = a.top2 ? g2 : g1, out = a.top2 ? g3 : g2;
        const bool unsure = lane < a.groups && (sum != sum || (out >> 9 > 1u &&
                            static_cast<float>((in >> 9) - (out >> 9)) <= delta * fine + 2.f));
        if (!__any_sync(0xFFFFFFFFu, unsure)) {
          int rank = 0;
          for (int g = 0; g < a.groups; ++g) {
            const double other = __shfl_sync(0xFFFFFFFFu, sum, g);
            rank += other > sum || (other == sum && g < lane) ? 1 : 0;
          }
          const uint32_t in_set = __ballot_sync(0xFFFFFFFFu, lane < a.groups && rank < a.topk_groups);
          kept = group < a.groups && (in_set >> group & 1u);
          close = false;
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (!kept) key[i] = 0u;
    }
    uint32_t mine = 0u;  // lane j: the (j+1)-th key
    for (int r = 0; r <= a.k; ++r) {
      const uint32_t best = __reduce_max_sync(0xFFFFFFFFu, key[0]);
      if (lane == r) mine = best;
      if (key[0] == best) {  // one lane, or none left anywhere
#pragma unroll
        for (int i = 0; i + 1 < V; ++i) key[i] = key[i + 1];
        key[V - 1] = 0u;
      }
    }
    int id = mine != 0u ? 511 - static_cast<int>(mine & 511u) : -1;
    float xs = id >= 0 ? to_float(p[id]) : -INFINITY;
    {
      const float bs = id >= 0 && a.bias != nullptr ? __ldg(a.bias + id) : 0.f;
      const uint32_t order = mine >> 9;
      const float cs = order > 1u ? (LOGIT ? xs : quick_score(softmax, xs, sc.top, inv) + bs) : -INFINITY;
      const uint32_t on = __shfl_down_sync(0xFFFFFFFFu, order, 1);
      const float cn = __shfl_down_sync(0xFFFFFFFFu, cs, 1);
      const float xn = __shfl_down_sync(0xFFFFFFFFu, xs, 1);
      const float bn = __shfl_down_sync(0xFFFFFFFFu, bs, 1);
      const bool same = xs == xn && bs == bn;
      const bool chosen = lane < a.k && on > 1u;  // experts that are off stand in their order
      bool again = close;
      if constexpr (LOGIT) {
        if (!kExact)
          again |= __any_sync(0xFFFFFFFFu, chosen && order == on && (!same || lane == a.k - 1));
      } else {
        const bool near = __any_sync(0xFFFFFFFFu, chosen && !(cs - cn > delta) && !same);
        const bool tie = __shfl_sync(0xFFFFFFFFu, chosen && same ? 1 : 0, a.k - 1) != 0;
        if (near || tie) {
          // Experts that could belong before the k-th, apart from its equals.
          const float ck = __shfl_sync(0xFFFFFFFFu, cs, a.k - 1);
          const float xk = __shfl_sync(0xFFFFFFFFu, xs, a.k - 1);
          const float bk = __shfl_sync(0xFFFFFFFFu, bs, a.k - 1);
          // In the upper half its equals themselves, which matter where one
          // of the choices before it may belong behind it.
          int rivals = 0;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float c = x[i] > -INFINITY ? quick_score(softmax, x[i], sc.top, inv) + bias[i] : -INFINITY;
            if (kept && i < count && !(c <= ck - delta) && c > -INFINITY)
              rivals += x[i] == xk && bias[i] == bk ? 1 << 16 : 1;
          }
          const int all = static_cast<int>(__reduce_add_sync(0xFFFFFFFFu, rivals));
          const bool known = lane <= a.k && order > 1u && !(cs <= ck - delta);
          const bool equal = xs == xk && bs == bk;
          const uint32_t found = __ballot_sync(0xFFFFFFFFu, known && !equal);
          const uint32_t equals = __ballot_sync(0xFFFFFFFFu, known && equal);
          const bool behind = __any_sync(0xFFFFFFFFu, known && lane < a.k && !equal && !(cs > ck + delta));
          again |= softmax || (all & 0xFFFF) > __popc(found) || (behind && all >> 16 > __popc(equals));
          if (near && !again) {
            // These k + 1 in the order of their fp64 choices.
            double exact = -INFINITY;
            if (order > 1u) exact = score_of<double>(softmax, xs, Scale<double>{0.0, 1.0}) + bs;
            int rank = 0;
            for (int r = 0; r <= a.k; ++r) {
              const double other = __shfl_sync(0xFFFFFFFFu, exact, r);
              const int oid = __shfl_sync(0xFFFFFFFFu, id, r);
              rank += oid >= 0 && (id < 0 || other > exact || (other == exact && oid < id)) ? 1 : 0;
            }
            const int was = id;
            const float x_was = xs;
            for (int r = 0; r <= a.k; ++r) {
              const uint32_t who = __ballot_sync(0xFFFFFFFFu, lane <= a.k && was >= 0 && rank == r);
              const int src = who ? __ffs(who) - 1 : 0;
              const int i = __shfl_sync(0xFFFFFFFFu, was, src);
              const float v = __shfl_sync(0xFFFFFFFFu, x_was, src);
              if (lane == r) id = who ? i : -1, xs = v;
            }
          }
        }
      }
      if (again) {  // the same in every lane
        float copy[V];  // its address leaves this function: x stays in registers
#pragma unroll
        for (int i = 0; i < V; ++i) copy[i] = x[i];
        id = order_row_exactly<V>(a, copy, valid, first);
        xs = id >= 0 ? to_float(p[id]) : -INFINITY;
      }
    }
    float w = 0.f;
    if (!softmax && __any_sync(0xFFFFFFFFu, lane < a.k && xs < -80.f && xs > -INFINITY)) {
      w = far_sigmoid_weight(xs, lane < a.k, a.renorm != 0, a.scale);
    } else {
      if (softmax && a.renorm) {
        // Relative to the largest chosen logit: the row's sum cancels, and the
        // chosen cannot all underflow.
        const float t = warp_max(lane < a.k ? xs : -INFINITY);
        if (lane < a.k && t > -INFINITY) w = expf(xs - t);
        bool poison = false;  // a NaN or +inf anywhere in the row makes every score NaN
#pragma unroll
        for (int i = 0; i < V; ++i) poison |= i < count && !(x[i] < INFINITY);
        if (__any_sync(0xFFFFFFFFu, poison)) w = __int_as_float(0x7FC00000);
      } else if (lane < a.k) {
        w = sc.sum == 0.f ? 0.f : score_of<float>(softmax, xs, sc);  // 0: a row with nothing on
      }
      if (a.renorm) {
        const float total = warp_total(lane < a.k ? w : 0.f);
        w = total == 0.f ? 0.f : w / total;
      }
      w *= a.scale;
    }
    if (lane < a.k) {
      a.w[row * a.k + lane] = w;
      a.ids[row * a.k + lane] = id;
    }
  }
}

using RouteKernel = void (*)(RouteArgs);

template <typename T, RouteBy BY>
static RouteKernel route_kernel_of(int v) {
  switch (v) {
    case 1: return &k_route<T, 1, BY>;
    case 2: return &k_route<T, 2, BY>;
    case 4: return &k_route<T, 4, BY>;
    case 8: return &k_route<T, 8, BY>;
    case 16: return &k_route<T, 16, BY>;
    default: return &k_route<T, 32, BY>;
  }
}
template <typename T>
static RouteKernel route_kernel(int v, RouteBy by) {
  return by == kByLogit     ? route_kernel_of<T, kByLogit>(v)
         : by == kBySigmoid ? route_kernel_of<T, kBySigmoid>(v)
                            : route_kernel_of<T, kBySoftmax>(v);
}

}  // namespace arn
