// e4m3 quantisation with a power-of-two scale per block of 128, shared by the
// quantiser, the quantising dispatch and the SwiGLU product's epilogue.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include <type_traits>

namespace gf {

// bits of |v|, 0 for infinities and NaN: ordered as the finite magnitudes are,
// so that a block's largest magnitude is an integer maximum
__device__ __forceinline__ uint32_t finite_mag_bits(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
  return b < 0x7F800000u ? b : 0u;
}

// The scale of a block whose largest finite magnitude has the bits `mag`: the
// smallest power of two 2^e with mag <= 448 * 2^e. 448 = 1.75 * 2^8, so e is
// the magnitude's exponent - 8, plus one when its mantissa is above 1.75.
// e >= -126 keeps both 2^e and its reciprocal normal; a zero block has scale 1.
__device__ __forceinline__ float e4m3_scale(uint32_t mag, float& inv) {
  if (mag == 0u) {
    inv = 1.0f;
    return 1.0f;
  }
  int e = static_cast<int>(mag >> 23) - 8 + ((mag & 0x7FFFFFu) > 0x600000u ? 1 : 0);  // biased
  e = e < 1 ? 1 : e;
  inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
  return __uint_as_float(static_cast<uint32_t>(e) << 23);
}

// Two values times inv, rounded to nearest even e4m3 (lo in the low byte).
// Finite values are at most 448 after scaling; the conversion would saturate
// infinities, which become NaN here (x * 0 is NaN for infinities and NaN).
// FINITE: the caller knows that there are none.
template <bool FINITE = false>
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi, float inv) {
  lo = FINITE ? lo * inv : fmaf(lo, inv, lo * 0.0f);
  hi = FINITE ? hi * inv : fmaf(hi, inv, hi * 0.0f);
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

template <bool FINITE = false>
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d, float inv) {
  return e4m3x2<FINITE>(a, b, inv) | (e4m3x2<FINITE>(c, d, inv) << 16);
}

// 16-bit element pairs of a 32-bit word <-> floats
template <typename T>
struct Pair16;
template <>
struct Pair16<__half> {
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float one(__half h) { return __half2float(h); }
  static __device__ __forceinline__ __half round(float f) { return __float2half_rn(f); }
};
template <>
struct Pair16<__nv_bfloat16> {
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float one(__nv_bfloat16 h) { return __bfloat162float(h); }
  static __device__ __forceinline__ __nv_bfloat16 round(float f) { return __float2bfloat16_rn(f); }
};

// The largest magnitude's bits of 16-bit element pairs, in both halves of a word
// (two elements an instruction); FINITE: of the finite elements only.
template <typename T>
constexpr uint32_t kInf16 = std::is_same_v<T, __half> ? 0x7C00u : 0x7F80u;

template <typename T, bool FINITE = false>
__device__ __forceinline__ uint32_t max_mag2(uint32_t mag, const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t m = w[i] & 0x7FFF7FFFu;
    if (FINITE) m &= __vcmpltu2(m, kInf16<T> * 0x10001u);
    mag = __vmaxu2(mag, m);
  }
  return mag;
}

__device__ __forceinline__ uint32_t fold2(uint32_t mag2) { return max(mag2 & 0xFFFFu, mag2 >> 16); }

// the bits of a magnitude as fp32
template <typename T>
__device__ __forceinline__ uint32_t mag_to_f32(uint32_t mag) {
  return __float_as_uint(Pair16<T>::unpack(mag).x);
}

// 16 consecutive 16-bit elements (two 16-byte words)
template <typename T>
__device__ __forceinline__ void unpack16(const uint4& a, const uint4& b, float (&f)[16]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 v = Pair16<T>::unpack(w[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

// The scale of blocks of 128 elements, 16 in each of 8 consecutive lanes of a
// whole warp; `finite`: whether all of the lane's block are known to be.
// VOTE: the warp looks at all magnitudes first and once more at the finite ones
// where it found others, which spares the quantiser's instructions, 3 an
// element, that keep infinities and NaN apart (17408 x 5120 bf16: 44.0 us,
// without 45.7, with the maximum of floats 47.9). Not for the quantising
// dispatch, which HBM bounds with either: 40.8 us without the vote, 41.3 with.
template <typename T, bool VOTE>
__device__ __forceinline__ float block_scale16(const uint4& a, const uint4& b, float& inv,
                                               bool& finite) {
  auto largest = [&](auto only_finite) {
    constexpr bool kFinite = decltype(only_finite)::value;
    uint32_t mag = fold2(max_mag2<T, kFinite>(max_mag2<T, kFinite>(0u, a), b));
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, d));
    return mag;
  };
  uint32_t mag = largest(std::bool_constant<!VOTE>());
  finite = VOTE && mag < kInf16<T>;
  if (VOTE && !__all_sync(0xFFFFFFFFu, finite)) mag = largest(std::true_type());
  return e4m3_scale(mag_to_f32<T>(mag), inv);
}

template <bool FINITE = false>
__device__ __forceinline__ uint4 quant16(const float (&f)[16], float inv) {
  return make_uint4(e4m3x4<FINITE>(f[0], f[1], f[2], f[3], inv),
                    e4m3x4<FINITE>(f[4], f[5], f[6], f[7], inv),
                    e4m3x4<FINITE>(f[8], f[9], f[10], f[11], inv),
                    e4m3x4<FINITE>(f[12], f[13], f[14], f[15], inv));
}

// the 16 elements of two words in e4m3
template <typename T>
__device__ __forceinline__ uint4 quant_words(const uint4& a, const uint4& b, float inv,
                                             bool finite) {
  float f[16];
  unpack16<T>(a, b, f);
  return finite ? quant16<true>(f, inv) : quant16<false>(f, inv);
}

}  // namespace gf
