// A router's choice: scores of the experts from a token's logits, the best of the
// best groups, their weights; and the gradient of the logits.
//
//   s = softmax(l) or 1 / (1 + e^-l),  c = s + bias (no bias: the logits' own order)
//   groups by the sum of their 1 or 2 best c, experts by c, ties to the lowest index
//   weight = scale s (/ the sum of the token's chosen s)
//
// One warp a token: a lane holds consecutive experts of one group, so that lanes
// and experts are in the same order. Scores become order-preserving integers whose
// last bits are the place within the lane, so that a lane sorts its experts by
// minimum and maximum alone, a pick is one warp-wide integer maximum and the lowest
// lane that has it, and the lane that loses its best moves up the others. What bounds
// it is instructions (some 950 a token of 256 experts in groups with a bias: 16384 tokens
// 22 us; eight lanes a token, 128 experts of 16-bit logits: 250 and 7.2 us) and, for a
// token, latency (3 us).
//
// Experts are whole numbers, and scores may lie closer together than fp32, less the
// bits of the place, tells them apart. The comparisons that decide something are
// therefore looked at again: where two differ by no more than their error bounds, and
// not for equal inputs, those in question are compared in two fp32, and where that
// leaves it open in 64 bits (a few in a thousand tokens of 256 experts with a bias, and
// hardly any). Without a bias experts are compared by their logits; those of 16 bits
// leave the place's bits free and are exact at once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <limits.h>
#include <math.h>
#include <string.h>

#include <type_traits>

#include "block.h"
#include "ptx.cuh"
#include "two_float.cuh"

namespace gf {
namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
// Tokens from which on one may have eight lanes (us, a warp a token and eight lanes, bf16, logits in
// L2: 64 experts, 1536 tokens 2.75 and 2.42, 4096 3.7 and 2.5; 128 experts, 1024 tokens 2.8 and 3.0,
// 2048 3.1 and 3.05, 4096 4.4 and 3.2).
constexpr int kManyTokens = 2048;
constexpr int kWarps = 4;      // tokens of a CTA
constexpr float kNoScore = -745.f;  // e to this is 0 in 64 bits
// Sum of the chosen sigmoid scores from which on they are taken as they are: scores with parts of
// more than 2^-106 in it are then normal numbers.
constexpr float kLowSum = 0x1p-20f;

__device__ __forceinline__ float as_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float as_float(float v) { return v; }

// Order-preserving integers of scores: NaN above everything (as it would spread:
// arithmetic leaves the positive one), -inf and what is not there below kNone. The
// last bits are taken by the place i in the lane, the first place the largest.
constexpr int kNone = static_cast<int>(0x80800000u);  // of the lowest finite value

__device__ __forceinline__ int ordered(int bits) { return bits ^ ((bits >> 31) & 0x7FFFFFFF); }

template <int MASK>
__device__ __forceinline__ int key_of(float v, int i) {
  return (ordered(__float_as_int(v + 0.f)) & ~MASK) | (MASK - i);  // (-0 becomes 0)
}
// the value, less the place's bits
template <int MASK>
__device__ __forceinline__ float value_of(int key) {
  if (key < kNone) return -INFINITY;
  return __int_as_float(ordered(key & ~MASK));
}

// largest first: Batcher's odd-even merge sort (1968)
template <int N>
__device__ __forceinline__ void sort_keys(int (&k)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const int a = k[i + j], b = k[i + j + q];
            k[i + j] = max(a, b);
            k[i + j + q] = min(a, b);
          }
}

// 1 / (1 + e^-l) without overflow, in the accuracy that the weights take
__device__ __forceinline__ float logistic(float l) {
  const float e = expf(-fabsf(l));
  return __fdividef(l >= 0.f ? 1.f : e, 1.f + e);
}
__device__ __forceinline__ double logistic(double l) {
  const double e = exp(-fabs(l));
  return (l >= 0. ? 1. : e) / (1. + e);
}

// A chosen score over one factor of them all, where their sum divides it: softmax's is
// e^(l - top) with the largest chosen logit, and so is, over 1 + e^l, sigmoid's where top is
// negative, as e^l itself may have few bits in fp32, or none.
__device__ __forceinline__ float part_of_chosen(const RouteParams& p, float l, float top) {
  if (!p.sigmoid) return expf(l - top);
  if (!(top < 0.f) || l == -INFINITY) return logistic(l);
  const Two x = two_of(l, -top);  // (70, rounded, moves e^70 by 2^-18)
  const float e = expf(x.h);
  return fmaf(e, x.l, e) / (1.f + expf(l));
}

// a score as it is compared in fp32: e^x by the hardware exponential and the
// hardware reciprocal, small results flushed
__device__ __forceinline__ float exp_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}
__device__ __forceinline__ float fast_logistic(float x) {
  const float e = exp_fast(-fabsf(x));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return (x >= 0.f ? 1.f : e) * r;
}
__device__ __forceinline__ float fast_score(const RouteParams& p, float x, float top, float inv) {
  return p.sigmoid ? fast_logistic(x) : exp_fast(x - top) * inv;
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

// The largest logit and the sum of softmax's exponentials in 64 bits, by a whole warp.
template <typename L>
__device__ __forceinline__ void exact_softmax(const RouteParams& p, const L* row, double& top,
                                              double& total) {
  const int lane = threadIdx.x & 31;
  top = -INFINITY;
  for (int e = lane; e < p.experts; e += 32) top = fmax(top, static_cast<double>(as_float(row[e])));
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) top = fmax(top, __shfl_xor_sync(kAll, top, d));
  if (top == -INFINITY) top = 0.;
  double sum = 0.;
#pragma unroll 4
  for (int e = lane; e < p.experts; e += 32) sum += exp(static_cast<double>(as_float(row[e])) - top);
  total = warp_sum(sum);
}

// ------------------------------------------------------ comparisons more closely
// Scores in two fp32, right to 2^-38 of the largest: enough for all but a few in a
// million of the comparisons that fp32 leaves open, at a third of the time of 64 bits.
struct Scale {
  float top;   // softmax: the largest logit, and what every exponential is multiplied by
  Two inv;
  float size;  // the largest score
};

template <typename L>
__device__ __forceinline__ Scale scale_closely(const RouteParams& p, const L* row) {
  Scale c = {0.f, {1.f, 0.f}, 1.f};
  if (p.sigmoid) return c;
  const int lane = threadIdx.x & 31;
  float top = -INFINITY;
  for (int e = lane; e < p.experts; e += 32) top = fmaxf(top, as_float(row[e]));
  top = warp_max(top);
  c.top = top == -INFINITY ? 0.f : top;
  Two sum = {0.f, 0.f};
#pragma unroll 2
  for (int e = lane; e < p.experts; e += 32) {
    const float l = as_float(row[e]);
    const Two x = two_of(c.top, -l);
    if (l != -INFINITY) sum = two_add(sum, two_exp_minus(x.h, x.l));
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1)
    sum = two_add(sum, Two{__shfl_xor_sync(kAll, sum.h, d), __shfl_xor_sync(kAll, sum.l, d)});
  c.inv = two_inverse(sum);
  c.size = c.inv.h;
  return c;
}

__device__ __forceinline__ Two score_closely(const RouteParams& p, const Scale& c, float l) {
  if (p.sigmoid) {
    const Two e = two_exp_minus(fabsf(l), 0.f);
    const Two q = two_inverse(two_add(e, 1.f));
    return l >= 0.f ? q : two_mul(e, q);
  }
  const Two x = two_of(c.top, -l);
  return two_mul(two_exp_minus(x.h, x.l), c.inv);
}

__device__ __forceinline__ bool above(const Two& a, const Two& b) {
  return a.h > b.h || (a.h == b.h && a.l > b.l);
}
// whether a is told from b (not where one is no number, or both are infinite)
__device__ __forceinline__ bool apart(const Two& a, const Two& b, float size) {
  return fabsf((a.h - b.h) + (a.l - b.l)) > size * 0x1p-37f + fabsf(a.h) * 0x1p-44f;
}

// Whether this lane's group is one of the best. Groups whose fp32 score lies between
// `low` and `high` are in question, the others keep theirs; of them only experts whose
// fp32 score is at least `least` may be among the two best. *sure: whether that decides.
template <typename L>
__device__ __noinline__ bool groups_closely(const RouteParams& p, const L* row, int base, int count,
                                            float score32, float low, float high, float least,
                                            float top32, float inv, bool* sure) {
  const int lane = threadIdx.x & 31;
  const bool by_logit = p.bias == nullptr && p.group_best == 1;
  const Scale scale = by_logit ? Scale{0.f, {1.f, 0.f}, 0.f} : scale_closely(p, row);
  const bool asked = !(score32 < low) && !(score32 > high);
  uint64_t left = 0ull;  // places of experts to look at
  for (int i = 0; i < count && asked; ++i) {
    const float l = as_float(row[base + i]);
    const float add = p.bias != nullptr ? p.bias[base + i] : 0.f;
    const float c32 = by_logit ? l : fast_score(p, l, top32, inv) + add;
    if (!(c32 < least) && c32 != -INFINITY && l != -INFINITY) left |= 1ull << i;
  }
  // the two best, and the logits and biases that they are of
  const Two kNone2 = {-INFINITY, 0.f};
  Two a = kNone2, b = kNone2;
  float la = 0.f, lb = 0.f, ba = 0.f, bb = 0.f;
  bool good = true;  // every score a number
  while (__any_sync(kAll, left != 0ull)) {
    if (left == 0ull) continue;
    const int i = __ffsll(static_cast<long long>(left)) - 1;
    left &= left - 1ull;
    const float l = as_float(row[base + i]), add = p.bias != nullptr ? p.bias[base + i] : 0.f;
    const Two c = by_logit ? Two{l, 0.f} : two_add(score_closely(p, scale, l), add);
    good = good && fabsf(c.h) < INFINITY;
    if (above(c, a)) {
      b = a, lb = la, bb = ba;
      a = c, la = l, ba = add;
    } else if (above(c, b)) {
      b = c, lb = l, bb = add;
    }
  }
  for (int d = 1; d < 1 << p.lane_shift; d <<= 1) {
    auto from = [&](float v) { return __shfl_xor_sync(kAll, v, d); };
    const Two oa = {from(a.h), from(a.l)}, ob = {from(b.h), from(b.l)};
    const float ola = from(la), olb = from(lb), oba = from(ba), obb = from(bb);
    // (of equal ones the lower lane's first, in both lanes)
    const bool mine = above(a, oa) || (!above(oa, a) && (lane & d) == 0);
    const Two less = mine ? oa : a, second = mine ? b : ob;
    const float lless = mine ? ola : la, bless = mine ? oba : ba;
    const float lsec = mine ? lb : olb, bsec = mine ? bb : obb;
    a = mine ? a : oa, la = mine ? la : ola, ba = mine ? ba : oba;
    const bool keep = above(second, less);
    b = keep ? second : less, lb = keep ? lsec : lless, bb = keep ? bsec : bless;
  }
  Two score = a;
  if (p.group_best == 2 && b.h != -INFINITY) score = two_add(a, b);
  if (p.group_best == 1) lb = bb = 0.f;
  if (!asked) score = {score32, 0.f};
  const int g = lane >> p.lane_shift;
  const int in_question = g < p.groups && asked ? 1 : 0;
  int rank = 0;
  uint32_t close = 0u;  // groups that this one is not told from
  for (int h = 0; h < p.groups; ++h) {
    const int src = h << p.lane_shift;
    const Two o = {__shfl_sync(kAll, score.h, src), __shfl_sync(kAll, score.l, src)};
    const float ola = __shfl_sync(kAll, la, src), olb = __shfl_sync(kAll, lb, src);
    const float oba = __shfl_sync(kAll, ba, src), obb = __shfl_sync(kAll, bb, src);
    const int other_in_question = __shfl_sync(kAll, in_question, src);
    const bool same = ola == la && olb == lb && oba == ba && obb == bb;
    const bool both = (other_in_question & in_question) != 0;
    if (h == g) continue;
    if (above(o, score) || (h < g && !above(score, o))) ++rank;
    if (both && !same && !apart(o, score, 2.f * scale.size)) close |= 1u << h;
  }
  const bool in = g < p.groups && rank < p.topk_groups;
  // (which decides nothing where both stay, or go)
  const uint32_t stay = __ballot_sync(kAll, in);
  for (int h = 0; h < p.groups; ++h)
    if ((close >> h & 1u) != 0u && ((stay >> (h << p.lane_shift) & 1u) != 0u) != in) good = false;
  *sure = __all_sync(kAll, good);
  return in;
}

// The order of up to 32 experts, one a lane (`expert` -1: none): returns the one of rank
// `lane`. *sure: whether that decides it.
template <typename L>
__device__ __noinline__ int order_closely(const RouteParams& p, const L* row, int expert, int n,
                                          bool* sure) {
  const int lane = threadIdx.x & 31;
  Scale scale = {0.f, {1.f, 0.f}, 0.f};
  if (p.bias != nullptr) scale = scale_closely(p, row);
  Two c = {-INFINITY, 0.f};
  float l = 0.f, add = 0.f;
  if (expert >= 0) {
    l = as_float(row[expert]);
    c = {l, 0.f};
    if (p.bias != nullptr) {
      add = p.bias[expert];
      c = two_add(score_closely(p, scale, l), add);
    }
  }
  bool good = expert < 0 || fabsf(c.h) < INFINITY;
  int rank = 0;
#pragma unroll 4
  for (int j = 0; j < n; ++j) {
    const Two o = {__shfl_sync(kAll, c.h, j), __shfl_sync(kAll, c.l, j)};
    const int e = __shfl_sync(kAll, expert, j);
    const float ol = __shfl_sync(kAll, l, j), oadd = __shfl_sync(kAll, add, j);
    const bool same = ol == l && oadd == add;
    if (e < 0 || expert < 0 || e == expert) continue;
    if (same ? e < expert : above(o, c)) ++rank;
    good = good && (same || apart(o, c, scale.size));
  }
  int out = -1;
#pragma unroll 4
  for (int j = 0; j < n; ++j) {
    const int where = __shfl_sync(kAll, rank, j), e = __shfl_sync(kAll, expert, j);
    if (where == lane && e >= 0) out = e;
  }
  *sure = __all_sync(kAll, good);
  return out;
}

// The choice of one token in 64 bits, by a whole warp: expert number j of it goes
// to slot j (lane j, or lane j - 32's second). Lane i looks after the experts i,
// i + 32, ..., and after group i.
template <typename L>
__device__ __noinline__ void choose_exactly(const RouteParams& p, const L* row, int& first,
                                            int& second) {
  const int lane = threadIdx.x & 31;
  double total = 1., top = 0.;
  if (!p.sigmoid) exact_softmax(p, row, top, total);
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

// CTAs of an SM (a warp a token: the grid is as large, warps loop over the tokens). With a
// warp a token fewer registers cost more than more warps gain: 60000 tokens, 256 experts
// in groups with a bias 66 us with 4, 75 with 6, 79 with 3; 128 experts in fp32 41 with 8,
// 48 with 6; 16384 tokens of 512 29.5 with 4, 31.5 with 3, 36 with 6.
constexpr int resident(int w, int vpl) {
  return w < 32 ? (vpl <= 8 ? 6 : 5) : vpl <= 4 ? 8 : vpl <= 16 ? 4 : 2;
}

// over the W lanes of a token
template <int W>
__device__ __forceinline__ int lanes_max(int v) {
  if constexpr (W == 32) {
    return __reduce_max_sync(kAll, v);
  } else {
#pragma unroll
    for (int d = W / 2; d >= 1; d >>= 1) v = max(v, __shfl_xor_sync(kAll, v, d));
    return v;
  }
}
template <int W>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int d = W / 2; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
  return v;
}
template <int W>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int d = W / 2; d >= 1; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}

// W lanes a token, VPL experts a lane. BIAS: scores are compared, else logits. Eight lanes
// a token: 16-bit logits that are compared as they are, of which nothing is ever in doubt.
template <typename L, int W, int VPL, bool BIAS>
__global__ void __launch_bounds__(32 * kWarps, resident(W, VPL))
    route_kernel(const __grid_constant__ RouteParams p) {
  constexpr int MASK = VPL - 1;
  constexpr int T = 32 / W;  // tokens of a warp
  // slots a lane: with a warp a token, the instances for more than 32 have two
  constexpr int S = W < 32 || VPL >= 32 ? 2 : 1;
  // keys tell everything apart but what is equal
  constexpr bool kExact = !BIAS && sizeof(L) == 2;
  // what the place's bits take from a value, relative to it
  constexpr float kCut = 1.2e-7f * VPL;
  static_assert(W == 32 || kExact, "no doubt with fewer lanes");
  // a token's lanes each have a sorted list: short ones in registers, others in shared memory
  constexpr bool kListed = W < 32 && VPL > 8;
  grid_dep_wait();
  grid_dep_launch();
  // the lane among its token's, and the token among its warp's
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & (W - 1), part = (threadIdx.x & 31) / W;
  __shared__ int2 slot_of[kWarps * T][W * S + 2];
  __shared__ int list_of[kListed ? 32 * kWarps : 1][VPL + 1];
  int2* slots = slot_of[warp * T + part];
  int* list = list_of[kListed ? threadIdx.x : 0];
  const uint32_t below = (1u << lane) - 1u;
  auto votes = [&](bool v) {
    const uint32_t b = __ballot_sync(kAll, v);
    return W == 32 ? b : b >> (W * part) & ((1u << (W & 31)) - 1u);
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps * T;
  int64_t token = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * T + part;
  if (token - part >= p.tokens) return;
  // this lane's experts
  const int g = lane >> p.lane_shift, lane_mask = (1 << p.lane_shift) - 1;
  const int in_group = (lane & lane_mask) * p.per_lane;
  const int base = g * p.group_size + in_group;
  const int experts_here = g < p.groups ? max(0, min(p.per_lane, p.group_size - in_group)) : 0;
  int count = token < p.tokens ? experts_here : 0;
  float bias[BIAS ? VPL : 1];
  if constexpr (BIAS) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) bias[i] = i < count ? p.bias[base + i] : 0.f;
  }
  const bool grouped = p.groups > 1;
  const bool sums = grouped && p.group_best == 2;
  const int picks = p.topk + (kExact ? 0 : 1);  // the next one, to compare the last with

  float l[VPL];
  load_logits<L, VPL>(p, static_cast<const L*>(p.logits) + token * p.ld, base, count, l);
  for (;;) {
    const L* row = static_cast<const L*>(p.logits) + token * p.ld;
    // the largest logit, and the sum that all scores are divided by
    float top = 0.f, inv = 1.f;
    if (!p.sigmoid) {
      float m = l[0];
#pragma unroll
      for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);  // (of those that are numbers)
      if (m != m) m = -INFINITY;
      m = __int_as_float(ordered(lanes_max<W>(ordered(__float_as_int(m + 0.f)))));
      top = m == -INFINITY ? 0.f : m;
      if (BIAS || sums || !p.renorm) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) sum += exp_fast(l[i] - top);
        sum = lanes_sum<W>(sum);
        inv = sum == 0.f ? 0.f : 1.f / sum;  // (no logit above -inf: no scores)
      }
    }
    // the error of fast_score: of the exponential (2^-22 of it and 2^-23 |x|), the sum
    // and the division. |x| e^x <= 0.4 bounds it by a part of the largest score, which
    // is `inv` for softmax and 1 for sigmoid.
    const float error = p.sigmoid ? 6e-7f : inv * (1.1e-6f + VPL * 6e-8f);
    int key[VPL];
    if constexpr (BIAS) {
      float c[VPL];
      if (p.sigmoid) {  // (one branch for all experts)
#pragma unroll
        for (int i = 0; i < VPL; ++i) c[i] = fast_logistic(l[i]);
      } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) c[i] = exp_fast(l[i] - top) * inv;
      }
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        key[i] = key_of<MASK>(l[i] == -INFINITY ? -INFINITY : c[i] + bias[i], i);  // (c may be NaN)
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = key_of<MASK>(l[i], i);
    }
    // the two largest logits with all their bits: e^l takes a cut of l, which may be far from
    // 0, as a factor
    int first = INT_MIN, second = INT_MIN;
    if constexpr (!BIAS && !kExact) {
      if (sums) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const int k = ordered(__float_as_int(l[i] + 0.f));
          second = max(second, min(first, k));
          first = max(first, k);
        }
      }
    }
    sort_keys<VPL>(key);
    bool out = false, unsure = false;  // this lane's group goes; the choice needs 64 bits
    if (grouped) {
      // the group's two best, over this lane's experts and then its lanes
      float a, b;
      if (!BIAS && sums) {  // sums are of scores, in which the experts are in the same order
        if constexpr (kExact) {
          first = key[0] & ~MASK;
          second = VPL > 1 ? key[VPL > 1 ? 1 : 0] & ~MASK : INT_MIN;
        }
        a = fast_score(p, __int_as_float(ordered(first)), top, inv);
        b = fast_score(p, __int_as_float(ordered(second)), top, inv);
        if (first < kNone) a = -INFINITY;
        if (second < kNone) b = -INFINITY;
      } else {
        a = value_of<MASK>(key[0]);
        b = VPL > 1 ? value_of<MASK>(key[VPL > 1 ? 1 : 0]) : -INFINITY;
      }
      int ka = ordered(__float_as_int(a)), kb = ordered(__float_as_int(b));
      for (int d = 0; d < p.lane_shift; ++d) {
        const int oa = __shfl_xor_sync(kAll, ka, 1 << d), ob = __shfl_xor_sync(kAll, kb, 1 << d);
        kb = max(max(kb, ob), min(ka, oa));
        ka = max(ka, oa);
      }
      a = __int_as_float(ordered(ka));
      b = __int_as_float(ordered(kb));
      float score = a;
      if (sums && kb >= kNone) score += b;
      const int mine = g < p.groups ? ordered(__float_as_int(score + 0.f)) : INT_MIN;
      // the groups before this one, shared by the group's lanes
      int rank = 0;
      for (int h0 = 0; h0 < p.groups; h0 += lane_mask + 1) {
        const int h = h0 + (lane & lane_mask);
        const int other = __shfl_sync(kAll, mine, (h << p.lane_shift) & (W - 1), W);
        rank += h < p.groups && (other > mine || (other == mine && h < g)) ? 1 : 0;
      }
      for (int d = 0; d < p.lane_shift; ++d) rank += __shfl_xor_sync(kAll, rank, 1 << d);
      bool in = g < p.groups && rank < p.topk_groups;
      if (W == 32 && (!kExact || sums)) {
        // the worst group that stays and the best that goes
        const int lo = __reduce_min_sync(kAll, in ? mine : INT_MAX);
        const int hi = __reduce_max_sync(kAll, in ? INT_MIN : mine);
        if (hi >= kNone) {
          // rounding errors, by the largest terms of any group
          const float terms = ka < kNone ? 0.f : fabsf(a) + (kb < kNone ? 0.f : fabsf(b));
          const float most = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(terms)));
          const float tol = (BIAS || sums ? 4.f * error + 3e-7f * most : 0.f) + kCut * most;
          const float worst = __int_as_float(ordered(lo)), first = __int_as_float(ordered(hi));
          if (!(worst - first > tol)) {
            bool sure;
            in = groups_closely<L>(p, row, base, count, score, first - tol, worst + tol,
                                   (sums ? b : a) - tol, top, inv, &sure);
            unsure = !sure;
          }
        }
      }
      out = !in;
    }
    if (out) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = INT_MIN;
    }

    int head = key[0], place = 0;
    if constexpr (kListed) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) list[i] = key[i];
      list[VPL] = INT_MIN;
    }

    // the picks, each put down by the lane that has it: key and expert
    __syncwarp();
    int found = 0;
    for (int j = 0; j < picks; ++j) {
      const int mine = head & ~MASK;
      const int best = lanes_max<W>(mine);
      const bool some = best >= kNone;
      if (W == 32 ? !some : !__any_sync(kAll, some)) break;
      const uint32_t have = votes(mine == best);
      if (some) ++found;
      if (some && mine == best && (have & below) == 0u) {
        slots[j] = make_int2(mine, base + (MASK - (head & MASK)));
        if constexpr (kListed) {
          head = list[++place];
        } else {
#pragma unroll
          for (int i = 0; i + 1 < VPL; ++i) key[i] = key[i + 1];
          key[VPL - 1] = INT_MIN;
          head = key[0];
        }
      }
    }
    __syncwarp();
    // the next token's logits come meanwhile
    const int64_t next = token + step;
    const bool valid = token < p.tokens, more = W == 32 && next < p.tokens;
    if (more) {
      count = next < p.tokens ? experts_here : 0;
      load_logits<L, VPL>(p, row + step * p.ld, base, count, l);
    }
    int expert[S];
    float value[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int j = lane + W * s;
      const int2 slot = j < found ? slots[j] : make_int2(INT_MIN, -1);
      expert[s] = slot.y;
      value[s] = __int_as_float(ordered(slot.x));
    }
    if constexpr (!kExact) {
      // each pick against the one after it
      bool doubt = false, edge = false;
      auto near = [&](float v, float n) {
        const float most = fmaxf(fabsf(v), fabsf(n));
        return !(v - n > (BIAS ? 2.f * error + 4e-7f * most : 0.f) + kCut * most);
      };
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int j = lane + W * s;
        if (j < p.topk && j + 1 < found) {
          const int2 follow = slots[j + 1];
          if (near(value[s], __int_as_float(ordered(follow.x)))) {
            bool same = __float_as_uint(as_float(row[expert[s]])) ==
                        __float_as_uint(as_float(row[follow.y]));
            if (BIAS) same = same && p.bias[expert[s]] == p.bias[follow.y];
            doubt |= !same;
            // equal inputs, but the one after them may belong before both
            edge |= j == p.topk - 1;
          }
        }
      }
      if (!unsure && __any_sync(kAll, doubt || edge)) {
        // the picks and the one after them, if the next is further away; else all over
        bool few = p.topk < 32;
        if (few && found > p.topk) {
          const int m = __reduce_max_sync(kAll, head & ~MASK);
          const float last = __shfl_sync(kAll, value[0], p.topk);
          few = m < kNone || !near(last, __int_as_float(ordered(m)));
        }
        if (few && !__any_sync(kAll, doubt)) {
          // nothing else comes near
        } else if (few) {
          bool sure;
          const int e = order_closely<L>(p, row, expert[0], p.topk + 1, &sure);
          if (sure) expert[0] = e;
          unsure = !sure;
        } else {
          unsure = true;
        }
      }
    }
    if constexpr (W == 32) {
      if (unsure) {
        int second;
        choose_exactly<L>(p, row, expert[0], second);
        if (S == 2) expert[S - 1] = second;
      }
    }
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (lane + W * s >= p.topk) expert[s] = -1;

    // the weights; renormalised they are ratios of the chosen scores alone, unless these are 0
    // in 64 bits too. (Divided, then scaled: scale over a small sum may be infinite.)
    float x[S], w[S];
#pragma unroll
    for (int s = 0; s < S; ++s) x[s] = expert[s] >= 0 ? as_float(row[expert[s]]) : -INFINITY;
    if (p.renorm) {
      float most = 0.f, sum = 0.f;
      bool none = false, low = p.sigmoid;
      auto add_parts = [&] {
        sum = 0.f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
          w[s] = expert[s] >= 0 && !(none && x[s] == x[s]) ? part_of_chosen(p, x[s], most) : 0.f;
          sum += w[s];
        }
        sum = lanes_sum<W>(sum);
      };
      if (p.sigmoid) {  // as they are, unless they are small
        add_parts();
        low = __any_sync(kAll, sum < kLowSum);
      }
      if (!p.sigmoid || low) {
        most = lanes_max<W>(fmaxf(x[0], x[S - 1]));
        // (a token's weights do not depend on those of its warp's others)
        if (p.sigmoid && !(sum < kLowSum)) most = 0.f;
        none = (p.sigmoid ? most : most - top) < kNoScore;
        add_parts();
      }
#pragma unroll
      for (int s = 0; s < S; ++s) {
        w[s] = sum == 0.f ? 0.f : __fdividef(w[s], sum) * p.scale;
        // a logit without a number (or infinite) makes every score NaN, chosen or not
        if (inv != inv) w[s] = inv;
      }
    } else {
#pragma unroll
      for (int s = 0; s < S; ++s)
        w[s] = (p.sigmoid ? logistic(x[s]) : expf(x[s] - top) * inv) * p.scale;
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int j = lane + W * s;
      if (valid && j < p.topk) {
        p.expert[token * p.topk + j] = expert[s];
        p.weight[token * p.topk + j] = expert[s] >= 0 ? w[s] : 0.f;
      }
    }
    if (!more) return;
    token = next;
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

// All but softmax without renormalisation, where only the chosen experts have a
// gradient: eight lanes a token, the row put together in shared memory in the logits' type
// and written a word at a time, of 16 bytes or what divides a row's (16384 tokens of 128
// experts 3.5 us; CTAs that loop 5.1). S: slots a lane.
template <typename L, int S, typename Word>
__global__ void __launch_bounds__(32 * kWarps)
    route_grad_sparse_kernel(const __grid_constant__ RouteParams p) {
  constexpr int W = 8, kPer = static_cast<int>(sizeof(Word) / sizeof(L));  // elements of a word
  extern __shared__ __align__(16) uint8_t grad_rows[];  // [tokens of the CTA][ld]
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & (W - 1), words = static_cast<int>(p.ld) / kPer;
  Word* mine = reinterpret_cast<Word*>(grad_rows) + (threadIdx.x / W) * words;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * (32 * kWarps / W) + threadIdx.x / W;
  const bool valid = token < p.tokens;
  const L* row = static_cast<const L*>(p.logits) + token * p.ld;
  // softmax: a logit that is no number, or infinite, and the largest of all
  float of_all = -INFINITY;
  bool number = true;
  if (!p.sigmoid && valid) {
    for (int w = lane; w * kPer < p.experts; w += W) {
      const Word v = reinterpret_cast<const Word*>(row)[w];
      L e[kPer];
      memcpy(e, &v, sizeof(Word));
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const float x = w * kPer + j < p.experts ? as_float(e[j]) : -INFINITY;
        of_all = fmaxf(of_all, x);
        number = number && x < INFINITY;
      }
    }
  }
  int expert[S];
  float x[S], g[S], s[S], rest[S];
  float of_chosen = -INFINITY;
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const int j = lane + W * i;
    expert[i] = -1;
    g[i] = s[i] = rest[i] = 0.f;
    x[i] = -INFINITY;
    if (valid && j < p.topk) {
      const int e = p.expert[token * p.topk + j];
      const float d = p.d_weight[token * p.topk + j];
      if (e >= 0 && e < p.experts) {
        expert[i] = e;
        g[i] = d;
        x[i] = as_float(row[e]);
        of_chosen = fmaxf(of_chosen, x[i]);
      }
    }
  }
  if (!p.sigmoid) number = lanes_max<W>(number ? 0 : 1) == 0;
#pragma unroll
  for (int i = 0; i < S; ++i) {
    if (p.sigmoid && expert[i] >= 0) {
      s[i] = logistic(x[i]);
      rest[i] = logistic(-x[i]);
    } else {
      rest[i] = 1.f;
    }
  }
  float dot = 0.f;
  if (p.renorm) {
    float sum = 0.f;
    if (p.sigmoid) sum = lanes_sum<W>(S == 2 ? s[0] + s[S - 1] : s[0]);
    if (!p.sigmoid || __any_sync(kAll, sum < kLowSum)) {
      float top = lanes_max<W>(of_chosen);
      if (p.sigmoid && !(sum < kLowSum)) top = 0.f;  // (whatever the warp's other tokens are)
      const bool none = p.sigmoid ? top < kNoScore : !(top - lanes_max<W>(of_all) >= kNoScore);  // (and where all are -inf)
#pragma unroll
      for (int i = 0; i < S; ++i)
        s[i] = expert[i] >= 0 && !(none && x[i] == x[i]) ? part_of_chosen(p, x[i], top) : 0.f;
      sum = lanes_sum<W>(S == 2 ? s[0] + s[S - 1] : s[0]);
    }
    // (divided before they are summed: an expert alone has 1, and no gradient)
#pragma unroll
    for (int i = 0; i < S; ++i) s[i] = sum == 0.f ? 0.f : s[i] / sum;
    dot = lanes_sum<W>(S == 2 ? g[0] * s[0] + g[S - 1] * s[S - 1] : g[0] * s[0]);
  }
  const L fill = to_logit<L>(number ? 0.f : NAN);  // where nothing was chosen
  for (int w = lane; w < words; w += W) {
    L e[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) e[j] = w * kPer + j < p.experts ? fill : to_logit<L>(0.f);
    Word v;
    memcpy(&v, e, sizeof(Word));
    mine[w] = v;
  }
  __syncwarp();
  // an expert's slots in order, by the first of them
  float v[S];
#pragma unroll
  for (int i = 0; i < S; ++i) v[i] = p.scale * s[i] * rest[i] * (g[i] - dot);
  float total[S];
  bool writes[S];
#pragma unroll
  for (int i = 0; i < S; ++i) {
    total[i] = 0.f;
    writes[i] = expert[i] >= 0;
  }
  for (int j = 0; j < p.topk; ++j) {
    const int from = j & (W - 1);
    const int e = __shfl_sync(kAll, S == 2 && j >= W ? expert[S - 1] : expert[0], from, W);
    const float add = __shfl_sync(kAll, S == 2 && j >= W ? v[S - 1] : v[0], from, W);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      if (e == expert[i]) {
        total[i] += add;
        if (j < lane + W * i) writes[i] = false;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < S; ++i)
    if (writes[i]) reinterpret_cast<L*>(mine)[expert[i]] = to_logit<L>(number ? total[i] : NAN);
  __syncwarp();
  if (valid) {
    Word* out = reinterpret_cast<Word*>(static_cast<L*>(p.d_logits) + token * p.ld);
    for (int w = lane; w < words; w += W) out[w] = mine[w];
  }
}

template <typename L>
__global__ void __launch_bounds__(32 * kWarps) route_grad_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ float rows[];  // [kWarps][experts]
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (token >= p.tokens) return;
  const L* row = static_cast<const L*>(p.logits) + token * p.ld;
  float* d = rows + warp * p.experts;
  const bool all = !p.sigmoid && !p.renorm;  // every expert's logit takes part
  float top = 0.f, inv = 1.f;  // renormalised: top is of the chosen
  bool none = false;  // the chosen scores are 0
  float rest_of = 0.f;  // the gradient where nothing was chosen: NaN with a score of NaN
  if (p.renorm) {
    float of_chosen = -INFINITY;
    for (int j = lane; j < p.topk; j += 32) {
      const int e = p.expert[token * p.topk + j];
      if (e >= 0 && e < p.experts) of_chosen = fmaxf(of_chosen, as_float(row[e]));
    }
    top = warp_max(of_chosen);
    none = top < kNoScore;
  }
  if (!p.sigmoid) {
    float of_all = -INFINITY;
    bool number = true;
    for (int e = lane; e < p.experts; e += 32) {
      const float x = as_float(row[e]);
      of_all = fmaxf(of_all, x);
      number &= x < INFINITY;
    }
    of_all = warp_max(of_all);
    if (!__all_sync(kAll, number)) rest_of = NAN;
    if (p.renorm)
      none = !(top - of_all >= kNoScore);  // (and where all are -inf)
    else
      top = of_all == -INFINITY ? 0.f : of_all;
  }
  if (all) {
    float sum = 0.f;
    for (int e = lane; e < p.experts; e += 32) {
      d[e] = expf(as_float(row[e]) - top);
      sum += d[e];
    }
    sum = warp_sum(sum);
    inv = sum == 0.f ? 0.f : 1.f / sum;  // (no logit above -inf: no scores)
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
        if (!p.renorm)
          s[i] = p.sigmoid ? logistic(x) : expf(x - top) * inv;
        else if (!(none && x == x))
          s[i] = part_of_chosen(p, x, top);
        rest[i] = p.sigmoid ? logistic(-x) : 1.f;
      }
    }
  }
  float dot = 0.f;
  if (p.renorm) {
    // (divided before they are summed: an expert alone has 1, and no gradient)
    const float sum = warp_sum(s[0] + s[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) s[i] = sum == 0.f ? 0.f : s[i] / sum;
    dot = warp_sum(g[0] * s[0] + g[1] * s[1]);
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
  for (int i = 0; i < 2; ++i) v[i] = p.scale * s[i] * rest[i] * (g[i] - dot);
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

// The lanes of w that share a group, a power of two, and the experts of each.
RouteParams map_lanes(RouteParams p, int w, int size) {
  p.lane_shift = 0;
  while (p.groups << (p.lane_shift + 1) <= w) ++p.lane_shift;
  const int lanes = 1 << p.lane_shift;
  p.per_lane = (p.group_size + lanes - 1) / lanes;
  const int bytes = p.per_lane * size, word = bytes < 16 ? bytes : 16;
  p.vector = (p.per_lane & (p.per_lane - 1)) == 0 && p.group_size == lanes * p.per_lane &&
                     (p.ld * size) % word == 0
                 ? 1
                 : 0;
  return p;
}

// The instance for a call, logits of `size` bytes: lanes a token, experts a lane; its CTAs and
// the tokens that each has at a time.
struct RouteShape {
  int w, vpl, tokens;
  int64_t ctas;
};

RouteShape route_shape(const RouteParams& args, int size) {
  RouteShape s = {32, 0, kWarps, 0};
  if (size == 2 && args.tokens >= kManyTokens && args.bias == nullptr && args.groups <= 8 && args.topk <= 16 &&
      (args.groups == 1 || args.group_best == 1) && map_lanes(args, 8, size).per_lane <= 16)
    s.w = 8;
  const int per_lane = map_lanes(args, s.w, size).per_lane;
  const int n = s.w == 32 && args.topk > 32 && per_lane < 32 ? 32 : per_lane;  // two slots a lane
  for (s.vpl = s.w == 32 ? 1 : 4; s.vpl < n;) s.vpl *= 2;
  s.tokens = kWarps * (32 / s.w);
  // A warp a token: as many CTAs as are resident at once, more tokens follow in their loop,
  // each loaded ahead (16384 tokens, 256 experts in groups with a bias, with six CTAs an
  // SM: 23.4 us; a CTA for every four tokens 26.1). Four tokens a warp: a CTA for every 16, as the loop's last
  // turn would leave many idle (128 experts, 16384 / 65536 tokens 7.1 / 16.1 us; in a
  // loop 9.3 / 25.1).
  const int64_t all = (static_cast<int64_t>(args.tokens) + s.tokens - 1) / s.tokens;
  const int64_t most = static_cast<int64_t>(args.sms) * resident(s.w, s.vpl);
  s.ctas = s.w < 32 || all < most ? all : most;
  return s;
}

template <typename L, int W, int VPL>
cudaError_t route_of(const RouteParams& p, int64_t ctas, cudaStream_t stream, int pdl) {
  const dim3 grid(static_cast<unsigned>(ctas)), block(32 * kWarps);
  if constexpr (W == 32) {
    if (p.bias != nullptr)
      return launch_pdl(route_kernel<L, W, VPL, true>, grid, block, 0, stream, pdl, p);
  }
  return launch_pdl(route_kernel<L, W, VPL, false>, grid, block, 0, stream, pdl, p);
}

template <typename L>
cudaError_t route(const RouteParams& args, cudaStream_t stream, int pdl) {
  const RouteShape s = route_shape(args, static_cast<int>(sizeof(L)));
  const RouteParams p = map_lanes(args, s.w, static_cast<int>(sizeof(L)));
  if constexpr (sizeof(L) == 2) {
    if (s.w == 8) {
      switch (s.vpl) {
        case 4: return route_of<L, 8, 4>(p, s.ctas, stream, pdl);
        case 8: return route_of<L, 8, 8>(p, s.ctas, stream, pdl);
        case 16: return route_of<L, 8, 16>(p, s.ctas, stream, pdl);
      }
      return cudaErrorInvalidValue;
    }
  }
  switch (s.vpl) {
    case 1: return route_of<L, 32, 1>(p, s.ctas, stream, pdl);
    case 2: return route_of<L, 32, 2>(p, s.ctas, stream, pdl);
    case 4: return route_of<L, 32, 4>(p, s.ctas, stream, pdl);
    case 8: return route_of<L, 32, 8>(p, s.ctas, stream, pdl);
    case 16: return route_of<L, 32, 16>(p, s.ctas, stream, pdl);
    case 32: return route_of<L, 32, 32>(p, s.ctas, stream, pdl);
    case 64: return route_of<L, 32, 64>(p, s.ctas, stream, pdl);
  }
  return cudaErrorInvalidValue;
}

template <typename L, typename Word>
cudaError_t route_grad_sparse(const RouteParams& p, size_t row_bytes, cudaStream_t stream, int pdl) {
  constexpr int kTokens = 32 * kWarps / 8;
  const int64_t all = (static_cast<int64_t>(p.tokens) + kTokens - 1) / kTokens;
  const dim3 grid(static_cast<unsigned>(all)), block(32 * kWarps);
  return p.topk <= 8 ? launch_pdl(route_grad_sparse_kernel<L, 1, Word>, grid, block,
                                  kTokens * row_bytes, stream, pdl, p)
                     : launch_pdl(route_grad_sparse_kernel<L, 2, Word>, grid, block,
                                  kTokens * row_bytes, stream, pdl, p);
}

template <typename L>
cudaError_t route_grad(const RouteParams& p, cudaStream_t stream, int pdl) {
  // rows of whole words, up to 2 KB
  const size_t row_bytes = static_cast<size_t>(p.ld) * sizeof(L);
  if ((p.sigmoid || p.renorm) && p.topk <= 16 && row_bytes % 4 == 0 && row_bytes <= 2048) {
    if (row_bytes % 16 == 0) return route_grad_sparse<L, uint4>(p, row_bytes, stream, pdl);
    if (row_bytes % 8 == 0) return route_grad_sparse<L, uint2>(p, row_bytes, stream, pdl);
    return route_grad_sparse<L, uint32_t>(p, row_bytes, stream, pdl);
  }
  const dim3 grid((static_cast<unsigned>(p.tokens) + kWarps - 1) / kWarps), block(32 * kWarps);
  return launch_pdl(route_grad_kernel<L>, grid, block,
                    static_cast<size_t>(kWarps) * p.experts * 4, stream, pdl, p);
}

}  // namespace

int64_t route_ctas(const RouteParams& p, int type, int* tokens) {
  const RouteShape s = route_shape(p, type == 2 ? 4 : 2);
  *tokens = s.tokens;
  return s.ctas;
}

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
