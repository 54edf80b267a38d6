// Numbers held as the unevaluated sum of two fp32, h + l with |l| at most half a
// unit in the last place of h: some 48 bits. Error-free addition: Knuth, The Art of
// Computer Programming 2, 4.2.2; products by the fused multiply-add's exact remainder.
#pragma once

namespace gf {

// a + b = s + e exactly
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
  s = __fadd_rn(a, b);
  const float z = __fsub_rn(s, a);
  e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, z)), __fsub_rn(b, z));
}

struct Two {
  float h, l;
};

__device__ __forceinline__ Two two_of(float a, float b) {
  Two r;
  two_sum(a, b, r.h, r.l);
  return r;
}
// (|a| at least |b|, or a zero)
__device__ __forceinline__ Two two_quick(float a, float b) {
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Two two_add(Two a, float b) {
  const Two s = two_of(a.h, b);
  return two_quick(s.h, __fadd_rn(s.l, a.l));
}
__device__ __forceinline__ Two two_add(Two a, Two b) {
  const Two s = two_of(a.h, b.h);
  return two_quick(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ Two two_mul(Two a, Two b) {
  const float p = __fmul_rn(a.h, b.h);
  float e = __fmaf_rn(a.h, b.h, -p);
  e = __fmaf_rn(a.h, b.l, e);
  e = __fmaf_rn(a.l, b.h, e);
  return two_quick(p, e);
}
// 1 / a: one Newton step from the fp32 reciprocal
__device__ __forceinline__ Two two_inverse(Two a) {
  const float q = __frcp_rn(a.h);
  const float r = __fmaf_rn(-q, a.l, __fmaf_rn(-q, a.h, 1.f));
  return two_quick(q, __fmul_rn(q, r));
}

// 2^(-j / 16)
__constant__ const float kRoots[16][2] = {
    {0x1.000000p+0f, 0x0.000000p+0f},   {0x1.ea4afap-1f, 0x1.52486cp-28f},
    {0x1.d5818ep-1f, -0x1.822dbcp-28f}, {0x1.c199bep-1f, -0x1.3d56b2p-28f},
    {0x1.ae89fap-1f, -0x1.a94b14p-27f}, {0x1.9c4918p-1f, 0x1.51f848p-28f},
    {0x1.8ace54p-1f, 0x1.15506ep-28f},  {0x1.7a1148p-1f, -0x1.829fd0p-26f},
    {0x1.6a09e6p-1f, 0x1.9fcef4p-27f},  {0x1.5ab07ep-1f, -0x1.5bd5ecp-28f},
    {0x1.4bfdaep-1f, -0x1.593abcp-26f}, {0x1.3dea64p-1f, 0x1.824684p-26f},
    {0x1.306fe0p-1f, 0x1.4636e2p-26f},  {0x1.2387a6p-1f, 0x1.ceac48p-26f},
    {0x1.172b84p-1f, -0x1.c15748p-28f}, {0x1.0b5586p-1f, 0x1.9f3122p-26f}};

// e^-(a + b) for a >= 0 and a much smaller b, to some 2^-40 of it; 0 below 2^-150.
// a = n ln2 / 16 + r, where n times the first two of the three parts of ln2 / 16 is exact
// (12 bits each); e^-r by its series, the first three terms in two fp32.
__device__ __forceinline__ Two two_exp_minus(float a, float b) {
  if (a > 104.f) return {0.f, 0.f};
  const float n = rintf(a * 23.083120f);
  const Two x1 = two_of(__fmaf_rn(n, -0x1.62ep-5f, a), __fmul_rn(n, -0x1.0cp-19f));
  const Two x = two_quick(-x1.h, -__fadd_rn(__fmaf_rn(n, 0x1.05c61p-33f, x1.l), b));
  const float p = __fmul_rn(x.h, x.h);
  const float pe = __fmaf_rn(__fmul_rn(2.f, x.h), x.l, __fmaf_rn(x.h, x.h, -p));
  float q = __fmaf_rn(x.h, 1.f / 720.f, 1.f / 120.f);
  q = __fmaf_rn(q, x.h, 1.f / 24.f);
  q = __fmaf_rn(q, x.h, 1.f / 6.f);
  q = __fmul_rn(q, __fmul_rn(p, x.h));
  const Two s2 = two_of(x.h, __fmul_rn(0.5f, p));
  const float low = __fadd_rn(__fadd_rn(s2.l, x.l), __fmaf_rn(0.5f, pe, q));
  Two s = two_quick(1.f, s2.h);
  s = two_quick(s.h, __fadd_rn(s.l, low));
  const int i = static_cast<int>(n);
  s = two_mul(s, {kRoots[i & 15][0], kRoots[i & 15][1]});
  const int k = i >> 4;  // at most 150: in two steps
  const float half = __int_as_float((127 - (k >> 1)) << 23), rest = __int_as_float((127 - (k - (k >> 1))) << 23);
  return {s.h * half * rest, s.l * half * rest};
}

}  // namespace gf
