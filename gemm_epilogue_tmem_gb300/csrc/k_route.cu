// A router's choice: scores of the experts from a token's logits, the best of the
// best groups, their weights; and the gradient of the logits.
//
//   s = softmax(l) or 1 / (1 + e^-l),  c = s + bias (no bias: the logits' own order)
//   groups by the sum of their 1 or 2 best c, experts by c, ties to the lowest index
//   weight = scale s (/ the sum of the token's chosen s)
//
// One warp a token: a lane holds consecutive experts of one group, so that lanes
// and experts are in the same order and the lowest lane that has the maximum has the
// lowest expert. Of each pick every lane takes part in one warp-wide integer
// maximum over order-preserving keys; only the lane that loses its best looks again.
//
// Experts are whole numbers, and scores may lie closer together than fp32 tells
// them apart. The fp32 comparisons that decide something are therefore looked at
// again: where two differ by no more than their error bounds, and not for equal
// inputs, the token is chosen anew in 64 bits. Without a bias, experts are compared
// by their logits, exactly.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "block.h"
#include "ptx.cuh"

namespace gf {
namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kMaxSlots = 64;  // two a lane
constexpr int kWarps = 4;      // tokens of a CTA
constexpr float kNoScore = -745.f;  // e to this is 0 in 64 bits

__device__ __forceinline__ float as_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float as_float(float v) { return v; }

// Order-preserving keys: NaN above everything (as it would spread), -inf 0.
__device__ __forceinline__ uint32_t key_of(float v) {
  if (v != v) return 0xFFFFFFFFu;
  if (v == -INFINITY) return 0u;
  const uint32_t b = __float_as_uint(v + 0.f);  // -0 is 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
// (of a key that is not 0 or NaN's)
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
__device__ __forceinline__ float value_or(uint32_t key) {
  return key == 0u ? -INFINITY : key == 0xFFFFFFFFu ? NAN : value_of(key);
}

// 1 / (1 + e^-l) without overflow, in the accuracy that the weights take
__device__ __forceinline__ float logistic(float l) {
  const float e = expf(-fabsf(l));
  return (l >= 0.f ? 1.f : e) / (1.f + e);
}
__device__ __forceinline__ double logistic(double l) {
  const double e = exp(-fabs(l));
  return (l >= 0. ? 1. : e) / (1. + e);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
  return v;
}

// order of 64-bit scores: NaN above everything, ties to the lower index; index -1: none
__device__ __forceinline__ bool before(double a, int ia, double b, int ib) {
  if (ib < 0) return ia >= 0;
  if (ia < 0) return false;
  const bool na = a != a, nb = b != b;
  if (na || nb) return na != nb ? na : ia < ib;
  return a > b || (a == b && ia < ib);
}
__device__ __forceinline__ void warp_best(double& v, int& i) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    const double ov = __shfl_xor_sync(kAll, v, d);
    const int oi = __shfl_xor_sync(kAll, i, d);
    if (before(ov, oi, v, i)) {
      v = ov;
      i = oi;
    }
  }
}

// The choice of one token in 64 bits, by a whole warp: expert number j of it goes
// to slot j (lane j, or lane j - 32's second). Lane i looks after the experts i,
// i + 32, ..., and after group i.
template <typename L>
__device__ __noinline__ void choose_exactly(const RouteParams& p, const L* row, int& first,
                                            int& second) {
  const int lane = threadIdx.x & 31;
  double total = 1., top = -INFINITY;
  if (!p.sigmoid) {
    for (int e = lane; e < p.experts; e += 32) top = fmax(top, static_cast<double>(as_float(row[e])));
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) top = fmax(top, __shfl_xor_sync(kAll, top, d));
    if (top == -INFINITY) top = 0.;
    double sum = 0.;
    for (int e = lane; e < p.experts; e += 32) sum += exp(static_cast<double>(as_float(row[e])) - top);
    total = warp_sum(sum);
  }
  auto score = [&](double l) { return p.sigmoid ? logistic(l) : exp(l - top) / total; };
  double c[32];  // of this lane's experts
  for (int i = 0; i < 32; ++i) {
    const int e = lane + 32 * i;
    c[i] = -INFINITY;
    if (e < p.experts) {
      const double l = as_float(row[e]);
      c[i] = l == -INFINITY ? l : p.bias != nullptr ? score(l) + static_cast<double>(p.bias[e]) : l;
    }
  }
  uint32_t kept = kAll;  // groups, a bit each
  if (p.groups > 1) {
    double mine = -INFINITY;  // this lane's group's score
    for (int g = 0; g < p.groups; ++g) {
      double a = -INFINITY, b = -INFINITY;  // the group's two best
      int ia = -1;
      for (int i = 0; i < 32; ++i) {
        const int e = lane + 32 * i;
        if (e >= p.experts || e / p.group_size != g) continue;
        const double l = as_float(row[e]);
        // (sums are of scores; one best may be compared as the experts are)
        const double v = p.bias != nullptr || p.group_best == 1 || l == -INFINITY ? c[i] : score(l);
        if (v == -INFINITY) continue;
        if (before(v, e, a, ia)) {
          b = a;
          a = v;
          ia = e;
        } else if (before(v, e, b, b == -INFINITY ? -1 : 0)) {
          b = v;
        }
      }
      double best = a;
      int who = ia;
      warp_best(best, who);
      double next = ia == who ? b : a;
      int ok = next == -INFINITY ? -1 : lane;
      warp_best(next, ok);
      double sum = who < 0 ? -INFINITY : best;
      if (p.group_best == 2 && who >= 0 && ok >= 0) sum += next;
      if (lane == g) mine = sum;
    }
    kept = 0u;
    for (int j = 0; j < p.topk_groups; ++j) {
      double v = mine;
      int g = lane < p.groups && !(kept >> lane & 1u) ? lane : -1;
      warp_best(v, g);
      kept |= 1u << g;
    }
  }
  uint32_t taken = 0u;  // this lane's experts, a bit each
  for (int i = 0; i < 32; ++i) {
    const int e = lane + 32 * i;
    if (e >= p.experts || c[i] == -INFINITY ||
        (p.groups > 1 && !(kept >> (e / p.group_size) & 1u)))
      taken |= 1u << i;
  }
  first = second = -1;
  for (int j = 0; j < p.topk; ++j) {
    double v = -INFINITY;
    int e = -1;
    for (int i = 0; i < 32; ++i) {
      if (!(taken >> i & 1u) && before(c[i], lane + 32 * i, v, e)) {
        v = c[i];
        e = lane + 32 * i;
      }
    }
    warp_best(v, e);
    if (e >= 0 && (e & 31) == lane) taken |= 1u << (e >> 5);
    if (lane == (j & 31)) (j < 32 ? first : second) = e;
  }
}

// This lane's logits: experts `first` .. `first` + per_lane - 1 of its group; -inf
// for those that are not there.
template <typename L, int VPL>
__device__ __forceinline__ void load_logits(const RouteParams& p, const L* row, int first, int count,
                                            float (&l)[VPL]) {
  constexpr int kBytes = VPL * static_cast<int>(sizeof(L));
  if constexpr (kBytes >= 4) {
    if (p.vector && count == VPL) {
      constexpr int kWord = kBytes >= 16 ? 16 : kBytes;
      constexpr int kPer = kWord / static_cast<int>(sizeof(L));
      using Word = std::conditional_t<kWord == 16, uint4, std::conditional_t<kWord == 8, uint2, uint32_t>>;
      const Word* at = reinterpret_cast<const Word*>(row + first);
#pragma unroll
      for (int i = 0; i < VPL / kPer; ++i) {
        const Word w = at[i];
        const L* e = reinterpret_cast<const L*>(&w);
#pragma unroll
        for (int j = 0; j < kPer; ++j) l[i * kPer + j] = as_float(e[j]);
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) l[i] = i < count ? as_float(row[first + i]) : -INFINITY;
}

template <typename L, int VPL>
__global__ void __launch_bounds__(32 * kWarps) route_kernel(const RouteParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (token >= p.tokens) return;
  const L* row = static_cast<const L*>(p.logits) + token * p.ld;
  // this lane's experts
  const int g = lane / p.lanes, in_group = (lane - g * p.lanes) * p.per_lane;
  const int base = g * p.group_size + in_group;
  int count = g < p.groups ? min(p.per_lane, p.group_size - in_group) : 0;
  if (count < 0) count = 0;
  float l[VPL];
  load_logits<L, VPL>(p, row, base, count, l);

  const bool bias = p.bias != nullptr;
  const bool grouped = p.groups > 1;
  const bool sums = grouped && p.group_best == 2;
  // the largest logit, and the sum that all scores are divided by
  float top = 0.f, inv = 1.f;
  if (!p.sigmoid) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
    top = value_or(__reduce_max_sync(kAll, m != m ? 0u : key_of(m)));  // (of those that are numbers)
    if (top == -INFINITY) top = 0.f;
    if (bias || sums || !p.renorm) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) sum += __expf(l[i] - top);
      inv = 1.f / warp_sum(sum);
    }
  }
  // scores as they are compared, and their error: of the exponential (2^-22 of it
  // and 2^-23 |x|), the sum and the division. |x| e^x <= 0.4 bounds the error by
  // a part of the largest score, which is `inv` for softmax and 1 for sigmoid.
  auto fast = [&](float x) {
    if (!p.sigmoid) return __expf(x - top) * inv;
    const float e = __expf(-fabsf(x));
    return __fdividef(x >= 0.f ? 1.f : e, 1.f + e);
  };
  const float error = p.sigmoid ? 6e-7f : inv * (1.1e-6f + VPL * 6e-8f);
  uint32_t key[VPL];
  bool doubt = false;
  if (bias || sums) {
    float c[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      c[i] = l[i] == -INFINITY ? l[i] : fast(l[i]);
      if (bias && i < count && l[i] != -INFINITY) c[i] += p.bias[base + i];
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = key_of(c[i]);
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = key_of(l[i]);
  }
  if (grouped) {
    // the group's two best, over this lane's experts and then its lanes
    uint32_t a = 0u, b = 0u;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      b = max(b, min(a, key[i]));
      a = max(a, key[i]);
    }
    for (int d = 1; d < p.lanes; d <<= 1) {
      const uint32_t oa = __shfl_xor_sync(kAll, a, d), ob = __shfl_xor_sync(kAll, b, d);
      b = max(max(b, ob), min(a, oa));
      a = max(a, oa);
    }
    float score = value_or(a);
    if (sums && b != 0u) score += value_or(b);
    const uint32_t mine = g < p.groups ? key_of(score) : 0u;
    int rank = 0;
    for (int h = 0; h < p.groups; ++h) {
      const uint32_t other = __shfl_sync(kAll, mine, h * p.lanes);
      rank += other > mine || (other == mine && h < g) ? 1 : 0;
    }
    const bool in = g < p.groups && rank < p.topk_groups;
    if (bias || sums) {
      // the worst group that stays and the best that goes
      const uint32_t lo = ~__reduce_max_sync(kAll, in ? ~mine : 0u);
      const uint32_t hi = __reduce_max_sync(kAll, in ? 0u : mine);
      if (hi != 0u) {
        // rounding errors of sums, by the largest terms of any group
        const float terms = a == 0u ? 0.f : fabsf(value_or(a)) + (b == 0u ? 0.f : fabsf(value_or(b)));
        const float most = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(terms)));
        doubt = !(value_or(lo) - value_or(hi) > 4.f * error + 3e-7f * most);
      }
    }
    if (sums && !bias) {  // the experts themselves by their logits
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = key_of(l[i]);
    }
    if (!in) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = 0u;
    }
  }

  // the picks; slot j is in lane j % 32
  int expert[2] = {-1, -1};
  uint32_t picked[2] = {0u, 0u};
  uint32_t best = 0u;
  int at = 0;
  auto look = [&]() {
    best = key[0];
    at = 0;
#pragma unroll
    for (int i = 1; i < VPL; ++i) {
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
    }
  };
  look();
  const int picks = p.topk + (bias ? 1 : 0);  // the next one, to compare the last with
  uint32_t after = 0u;
  int after_expert = -1;
  for (int j = 0; j < picks; ++j) {
    const uint32_t m = __reduce_max_sync(kAll, best);
    if (m == 0u) break;
    const int who = __ffs(__ballot_sync(kAll, best == m)) - 1;
    const int e = __shfl_sync(kAll, base + at, who);
    if (j < p.topk) {
      if (lane == (j & 31)) {
        if (j < 32) {
          expert[0] = e;
          picked[0] = m;
        } else {
          expert[1] = e;
          picked[1] = m;
        }
      }
    } else {
      after = m;
      after_expert = e;
    }
    if (lane == who) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i == at) key[i] = 0u;
      look();
    }
  }
  if (bias) {
    // each pick against the one after it
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int j = lane + 32 * s;
      uint32_t next = __shfl_down_sync(kAll, picked[s], 1);
      int next_e = __shfl_down_sync(kAll, expert[s], 1);
      if (s == 0) {
        const uint32_t k32 = __shfl_sync(kAll, picked[1], 0);
        const int e32 = __shfl_sync(kAll, expert[1], 0);
        if (lane == 31) {
          next = k32;
          next_e = e32;
        }
      }
      if (j == p.topk - 1) {
        next = after;
        next_e = after_expert;
      }
      if (j < p.topk && picked[s] != 0u && next != 0u) {
        const float v = value_or(picked[s]), n = value_or(next);
        if (!(v - n > 2.f * error + 2e-7f * (fabsf(v) + fabsf(n)))) {
          const bool same = __float_as_uint(as_float(row[expert[s]])) ==
                                __float_as_uint(as_float(row[next_e])) &&
                            p.bias[expert[s]] == p.bias[next_e];
          doubt |= !same;
        }
      }
    }
  }
  if (__any_sync(kAll, doubt)) choose_exactly<L>(p, row, expert[0], expert[1]);

  // the weights; softmax over the chosen alone where they are renormalised, unless
  // their scores are 0 in 64 bits too
  bool none = false;
  if (!p.sigmoid && p.renorm) {
    const float of_all = top;
    float m = -INFINITY;
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (expert[s] >= 0) m = fmaxf(m, as_float(row[expert[s]]));
    top = value_or(__reduce_max_sync(kAll, key_of(m)));
    none = top - of_all < kNoScore;
    if (top == -INFINITY) top = 0.f;
  }
  float w[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    w[s] = 0.f;
    if (expert[s] >= 0) {
      const float x = as_float(row[expert[s]]);
      w[s] = p.sigmoid ? logistic(x) : expf(x - top);
      if (!p.sigmoid && !p.renorm) w[s] *= inv;
    }
  }
  float factor = p.scale;
  if (p.renorm) {
    const float sum = warp_sum(w[0] + w[1]);
    // (chosen scores that are all 0 stay 0)
    factor = sum == 0.f || none ? 0.f : p.scale / sum;
    // a logit without a number (or infinite) makes every score NaN, chosen or not
    if (inv != inv) factor = inv;
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int j = lane + 32 * s;
    if (j < p.topk) {
      p.expert[token * p.topk + j] = expert[s];
      p.weight[token * p.topk + j] = w[s] * factor;
    }
  }
}

// ----------------------------------------------------------------- backward
// With p_j the part of slot j in the sum of the chosen scores, g its gradient:
//   renormalised: d s_j = scale / S (g_j - sum_i p_i g_i), else scale g_j
//   softmax:      d l = s (d s - sum_j s_j d s_j); renormalised the sum is 0, and
//                 s / S = e^(l - top) over their sum needs no other expert
//   sigmoid:      d l = d s  s (1 - s)
template <typename L>
__device__ __forceinline__ L to_logit(float v);
template <>
__device__ __forceinline__ __half to_logit<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 to_logit<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ float to_logit<float>(float v) { return v; }

template <typename L>
__global__ void __launch_bounds__(32 * kWarps) route_grad_kernel(const RouteParams p) {
  extern __shared__ float rows[];  // [kWarps][experts]
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (token >= p.tokens) return;
  const L* row = static_cast<const L*>(p.logits) + token * p.ld;
  float* d = rows + warp * p.experts;
  const bool all = !p.sigmoid && !p.renorm;  // every expert's logit takes part
  float top = 0.f, inv = 1.f;
  bool none = false;  // the chosen scores are 0
  float rest_of = 0.f;  // the gradient where nothing was chosen: NaN with a score of NaN
  if (!p.sigmoid) {
    float of_all = -INFINITY, of_chosen = -INFINITY;
    bool number = true;
    for (int e = lane; e < p.experts; e += 32) {
      const float x = as_float(row[e]);
      of_all = fmaxf(of_all, x);
      number &= x < INFINITY;
    }
    of_all = warp_max(of_all);
    if (!__all_sync(kAll, number)) rest_of = NAN;
    top = of_all;
    if (p.renorm) {
      for (int j = lane; j < p.topk; j += 32) {
        const int e = p.expert[token * p.topk + j];
        if (e >= 0 && e < p.experts) of_chosen = fmaxf(of_chosen, as_float(row[e]));
      }
      top = warp_max(of_chosen);
      none = top - of_all < kNoScore;
    }
    if (top == -INFINITY) top = 0.f;
  }
  if (all) {
    float sum = 0.f;
    for (int e = lane; e < p.experts; e += 32) {
      d[e] = expf(as_float(row[e]) - top);
      sum += d[e];
    }
    inv = 1.f / warp_sum(sum);
  } else {
    for (int e = lane; e < p.experts; e += 32) d[e] = rest_of;
  }
  int expert[2];
  float s[2], rest[2], g[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = lane + 32 * i;
    expert[i] = -1;
    s[i] = g[i] = rest[i] = 0.f;
    if (j < p.topk) {
      const int e = p.expert[token * p.topk + j];
      if (e >= 0 && e < p.experts) {
        expert[i] = e;
        g[i] = p.d_weight[token * p.topk + j];
        const float x = as_float(row[e]);
        s[i] = p.sigmoid ? logistic(x) : expf(x - top) * inv;
        rest[i] = p.sigmoid ? logistic(-x) : 1.f;
      }
    }
  }
  float factor = p.scale, dot = 0.f;
  if (p.renorm) {
    const float sum = warp_sum(s[0] + s[1]);
    const float part = sum == 0.f || none ? 0.f : 1.f / sum;
    dot = warp_sum(g[0] * s[0] + g[1] * s[1]) * part;
    factor = p.scale * part;
  } else if (all) {
    dot = warp_sum(g[0] * s[0] + g[1] * s[1]);
    __syncwarp();
    for (int e = lane; e < p.experts; e += 32) d[e] *= -(p.scale * dot * inv);
    dot = 0.f;
  }
  __syncwarp();
  // the slots' own terms; the same expert may be there twice: slot after slot, then
  float v[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) v[i] = factor * s[i] * rest[i] * (g[i] - dot);
  bool twice = false;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t peers = __match_any_sync(kAll, expert[i]);
    twice |= expert[i] >= 0 && (peers & (peers - 1u)) != 0u;
  }
  if (__any_sync(kAll, twice) || p.topk > 32) {
    for (int j = 0; j < p.topk; ++j) {
      const int e = __shfl_sync(kAll, j < 32 ? expert[0] : expert[1], j & 31);
      const float x = __shfl_sync(kAll, j < 32 ? v[0] : v[1], j & 31);
      if (lane == 0 && e >= 0) d[e] += x;
    }
  } else if (expert[0] >= 0) {
    d[expert[0]] += v[0];  // (NaN stays NaN)
  }
  __syncwarp();
  L* out = static_cast<L*>(p.d_logits) + token * p.ld;
  for (int64_t e = lane; e < p.ld; e += 32) out[e] = to_logit<L>(e < p.experts ? d[e] : 0.f);
}

template <typename L>
cudaError_t route(const RouteParams& p, cudaStream_t stream, int pdl) {
  const dim3 grid((p.tokens + kWarps - 1) / kWarps), block(32 * kWarps);
  const int n = p.per_lane;
  if (n <= 1) return launch_pdl(route_kernel<L, 1>, grid, block, 0, stream, pdl, p);
  if (n <= 2) return launch_pdl(route_kernel<L, 2>, grid, block, 0, stream, pdl, p);
  if (n <= 4) return launch_pdl(route_kernel<L, 4>, grid, block, 0, stream, pdl, p);
  if (n <= 8) return launch_pdl(route_kernel<L, 8>, grid, block, 0, stream, pdl, p);
  if (n <= 16) return launch_pdl(route_kernel<L, 16>, grid, block, 0, stream, pdl, p);
  if (n <= 32) return launch_pdl(route_kernel<L, 32>, grid, block, 0, stream, pdl, p);
  return launch_pdl(route_kernel<L, 64>, grid, block, 0, stream, pdl, p);
}

template <typename L>
cudaError_t route_grad(const RouteParams& p, cudaStream_t stream, int pdl) {
  const dim3 grid((p.tokens + kWarps - 1) / kWarps), block(32 * kWarps);
  return launch_pdl(route_grad_kernel<L>, grid, block,
                    static_cast<size_t>(kWarps) * p.experts * 4, stream, pdl, p);
}

}  // namespace

cudaError_t launch_route(const RouteParams& p, int type, cudaStream_t stream, int pdl) {
  switch (type) {
    case 0: return route<__half>(p, stream, pdl);
    case 1: return route<__nv_bfloat16>(p, stream, pdl);
    case 2: return route<float>(p, stream, pdl);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_route_grad(const RouteParams& p, int type, cudaStream_t stream, int pdl) {
  switch (type) {
    case 0: return route_grad<__half>(p, stream, pdl);
    case 1: return route_grad<__nv_bfloat16>(p, stream, pdl);
    case 2: return route_grad<float>(p, stream, pdl);
  }
  return cudaErrorInvalidValue;
}

}  // namespace gf
