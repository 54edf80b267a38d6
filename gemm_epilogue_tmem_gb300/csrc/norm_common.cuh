// What the norm's kernels share: sums, 16-bit elements.
//
//   r = round(x + residual),  y = r w rstd,  rstd = 1 / sqrt(mean(r^2) + eps)
//   g = d_y w,  d = rstd (g - r rstd^2 mean(g r)) + d_r,  d_w = sum of d_y r rstd
//
// e4m3 output: the scale of 128 elements is a power of two that the block's
// largest magnitude decides, so that a last bit of rstd could turn the whole block's
// scale. That magnitude is max|r w| rstd; the products r w of 16-bit values are exact
// in fp32, and where it matters rstd is held as the sum of two fp32, from a sum of
// squares held the same way and one Newton step, so that the scale is the one of 64-bit
// arithmetic.
#pragma once

#include <math.h>

#include <type_traits>

#include "block.h"
#include "fp8.cuh"
#include "ptx.cuh"
#include "two_float.cuh"

namespace gf {

// a sum of squares: fp32, or (EXACT) two fp32
template <bool EXACT>
struct Sum {
  float hi, lo;
  __device__ __forceinline__ void add(float v) {
    if constexpr (EXACT) {
      float e;
      two_sum(hi, v, hi, e);
      lo += e;
    } else {
      hi += v;
    }
  }
  __device__ __forceinline__ void add(const Sum& o) {
    add(o.hi);
    if constexpr (EXACT) lo += o.lo;
  }
  __device__ __forceinline__ Sum other(int lane_mask) const {
    Sum o = {0.f, 0.f};
    o.hi = __shfl_xor_sync(0xFFFFFFFFu, hi, lane_mask);
    if constexpr (EXACT) o.lo = __shfl_xor_sync(0xFFFFFFFFu, lo, lane_mask);
    return o;
  }
};

// 1 / sqrt(sum / n + eps), as hi + lo (EXACT)
template <bool EXACT>
__device__ __forceinline__ float inv_rms(const Sum<EXACT>& sum, int n, float eps, float& lo) {
  lo = 0.f;
  const float nf = static_cast<float>(n);
  if constexpr (!EXACT) {
    return rsqrtf(sum.hi / nf + eps);
  } else {
    float sh, sl;
    two_sum(sum.hi, sum.lo, sh, sl);
    if (!isfinite(sum.hi)) return rsqrtf(sum.hi);
    const float q = __fdiv_rn(sh, nf);
    const float ql = __fdiv_rn(__fadd_rn(__fmaf_rn(-q, nf, sh), sl), nf);
    float v, vl;
    two_sum(q, eps, v, vl);
    vl = __fadd_rn(vl, ql);
    const float r = rsqrtf(v);
    if (!isfinite(r)) return r;
    // r^2 and v r^2 with their rounding errors; 1 - v r^2 is small
    const float p = __fmul_rn(r, r), pe = __fmaf_rn(r, r, -p);
    const float t = __fmul_rn(v, p), te = __fmaf_rn(v, p, -t);
    float e = __fsub_rn(__fsub_rn(1.f, t), te);
    e = __fsub_rn(e, __fmul_rn(v, pe));
    e = __fsub_rn(e, __fmul_rn(vl, p));
    lo = __fmul_rn(__fmul_rn(0.5f, r), e);
    return r;
  }
}

// The bits of the largest magnitude of a block's y, from that of its r w: the rounded
// product may lie on the border of two scales and the product above it.
__device__ __forceinline__ uint32_t exact_mag(float mag, float rstd, float lo) {
  const float top = __fmul_rn(mag, rstd);
  const float err = __fmaf_rn(mag, lo, __fmaf_rn(mag, rstd, -top));
  uint32_t bits = finite_mag_bits(top);
  if ((bits & 0x7FFFFFu) == 0x600000u && err > 0.f) ++bits;
  return bits;
}

// the backward's two sums: r^2, and (d_y w) r
struct Sum2 {
  float rr, gr;
  __device__ __forceinline__ void add(const Sum2& o) {
    rr += o.rr;
    gr += o.gr;
  }
  __device__ __forceinline__ Sum2 other(int lane_mask) const {
    Sum2 o;
    o.rr = __shfl_xor_sync(0xFFFFFFFFu, rr, lane_mask);
    o.gr = __shfl_xor_sync(0xFFFFFFFFu, gr, lane_mask);
    return o;
  }
};

template <typename T>
__device__ __forceinline__ void unpack(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = Pair16<T>::unpack(w[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

template <typename T>
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
  return make_uint4(Pair16<T>::pack(f[0], f[1]), Pair16<T>::pack(f[2], f[3]),
                    Pair16<T>::pack(f[4], f[5]), Pair16<T>::pack(f[6], f[7]));
}

// x + residual in 16 bits, one rounding
template <typename T>
__device__ __forceinline__ uint32_t add2(uint32_t a, uint32_t b) {
  if constexpr (std::is_same_v<T, __half>) {
    const __half2 v = __hadd2_rn(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __nv_bfloat162 v = __hadd2_rn(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                        *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}
template <typename T>
__device__ __forceinline__ uint4 add8(const uint4& a, const uint4& b) {
  return make_uint4(add2<T>(a.x, b.x), add2<T>(a.y, b.y), add2<T>(a.z, b.z), add2<T>(a.w, b.w));
}

// Many rows of whole 16-byte words: the streaming kernels take them, see k_norm_stream.cu.
// Rows that a thread goes through at most, so that fp32 adds up no more terms of the weight's
// gradient in a row: beside the sum of 2^18 of its size a term has 6 bits left. More rows take more
// CTAs than are resident, each with sums of its own.
constexpr int64_t kMostTurns = 4096;

struct NormStream {
  int v, threads, rows;  // words a thread, threads a row, rows of a group
  int stages, ctas;
  size_t smem;
};
// (pairs: the threads have pairs of words)
bool norm_stream_shape(int64_t rows, int64_t hidden, int arrays, bool pairs, int sms, NormStream* s);
cudaError_t launch_norm_stream(const NormParams& p, const NormStream& s, int bf16,
                               cudaStream_t stream, int pdl);
cudaError_t launch_norm_grad_stream(const NormParams& p, const NormStream& s, int bf16,
                                    cudaStream_t stream, int pdl);

}  // namespace gf
