// What the block-scaled e4m3 kernels share: the table of groups and tiles,
// the tensor-core instruction and its descriptor, error reporting.
#pragma once

#include <type_traits>

#include "fp8.cuh"
#include "fp8_params.h"
#include "params.h"
#include "ptx.cuh"

namespace gf {

// One lane of a converged warp. The issuing warps run their loops with all
// lanes, so that stages, phases and descriptors are the warp's (uniform
// registers), and predicate the instructions themselves on the elected lane:
// issued from a branch that one lane took, the four instructions of a k-block
// cost enough others that the two epilogue warps on the same scheduler held
// them up (750 instead of 512 cycles a block).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e;
}

// D[tmem] (+)= A[smem desc] x B[smem desc], kind::f8f6f4 (8-bit in, fp32 acc),
// where `e`; PAIR: over a CTA pair.
template <bool PAIR>
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t accumulate, uint32_t e) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(e)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(e)
        : "memory");
}

// Arrive once on `bar` (PAIR: in both CTAs of the pair) when the products
// issued so far by the elected lane have completed, where `e`.
template <bool PAIR>
__device__ __forceinline__ void umma_commit_f8(uint32_t bar, uint32_t e) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster"
        ".b64 [%0], %1;\n\t}" ::"r"(bar),
        "h"(static_cast<uint16_t>(3)), "r"(e)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            bar),
        "r"(e)
        : "memory");
}

// 2-D tiled load where `e`; PAIR: signalled on a barrier of the pair (cluster
// address).
template <bool PAIR>
__device__ __forceinline__ void tma_load_f8(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int32_t x, int32_t y, uint32_t e) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
        ".mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(e)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(e)
        : "memory");
}

// Instruction descriptor, kind::f8f6f4: D fp32, A and B e4m3 (format 0), both
// K-major, N >> 3 at [17,23), M >> 4 at [24,29).
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ void fp8_raise(const Fp8Params& p, volatile int* abort_flag,
                                          int code) {
  *abort_flag = 1;
  atomicOr(p.status, code);
}

// acc += v * s, two columns at a time
__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t v0, uint32_t v1, uint64_t s) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(v0), "r"(v1));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(s));
}

__device__ __forceinline__ uint64_t both(float s) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %1};" : "=l"(v) : "f"(s));
  return v;
}

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}

__device__ __forceinline__ float2 split2(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}

// asynchronous 4-byte copy to shared memory (zero where !in), and an arrival
// on `bar` when this thread's copies so far have landed
__device__ __forceinline__ void cp_async_4(uint32_t dst, const float* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 4 : 0)
               : "memory");
}

__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// First row of group g (g == groups: the rows of no group, up to M). The
// offsets are the caller's device data: each is bounded to [the one before,
// M], so that whatever they hold every row index stays inside the matrices.
struct GroupTable {
  int32_t* row0;   // [groups + 2], row0[groups + 1] = M
  int32_t* tile0;  // [groups + 2], first tile of each group; the last: all tiles
};

// Fills the table (shared memory) with tiles of `tile_rows` rows x
// p-columns/`tile_cols` column tiles; called by all threads of the CTA, ends
// with a barrier. Warp 0 scans 32 groups at a time.
__device__ __forceinline__ void build_group_table(const Fp8Params& p, const GroupTable& g,
                                                  int tile_rows, int col_tiles) {
  if (threadIdx.x < 32) {
    const int lane = static_cast<int>(threadIdx.x);
    const int total = p.groups + 1;  // with the rows of no group
    int row_carry = 0, tile_carry = 0;
    for (int g0 = 0; g0 < total; g0 += 32) {
      const int i = g0 + lane;
      // the end of group i, not before any earlier end and at most M
      int end = 0;
      if (i < total)
        end = i == p.groups || p.offsets == nullptr ? p.M : min(max(p.offsets[i + 1], 0), p.M);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, end, d);
        if (lane >= d) end = max(end, v);
      }
      end = max(end, row_carry);
      int start = __shfl_up_sync(0xFFFFFFFFu, end, 1);
      if (lane == 0) start = row_carry;
      // rows before offsets[0] belong to no group; offsets start at 0
      int tiles = i < total ? (end - start + tile_rows - 1) / tile_rows * col_tiles : 0;
      const int own = tiles;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, tiles, d);
        if (lane >= d) tiles += v;
      }
      if (i < total) {
        g.row0[i] = start;
        g.tile0[i] = tile_carry + tiles - own;
      }
      row_carry = __shfl_sync(0xFFFFFFFFu, end, 31);
      tile_carry += __shfl_sync(0xFFFFFFFFu, tiles, 31);
    }
    if (lane == 0) {
      g.row0[total] = p.M;
      g.tile0[total] = tile_carry;
    }
  }
  __syncthreads();
}

// the group that tile t < tile0[groups + 1] belongs to
__device__ __forceinline__ int group_of_tile(const GroupTable& g, int groups, int t) {
  int lo = 0, hi = groups + 1;  // tile0[lo] <= t < tile0[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (g.tile0[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// silu(g) u = g u / (1 + 2^(-g log2 e)), with the hardware's exponential and
// reciprocal (relative errors of 2^-22 and 2^-23): the result is rounded to
// e4m3. Below g = -87 the reciprocal is flushed to the limit 0.
__device__ __forceinline__ float silu_mul(float g, float u) {
  float t, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + t));
  return g * r * u;
}

// The SwiGLU of a thread's 64 gate (acc[0..31], two a register pair) and up
// columns (acc[32..63]), in place of the gate; columns from `valid` on are zero.
// Returns the largest finite magnitude's bits; `finite`: whether all are.
__device__ __forceinline__ uint32_t swiglu64(uint64_t (&acc)[64], int valid, bool& finite) {
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const float2 g = split2(acc[j]), u = split2(acc[32 + j]);
    acc[j] = pack2(silu_mul(g.x, u.x), silu_mul(g.y, u.y));
  }
  if (valid < 64) {
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const float2 h = split2(acc[j]);
      acc[j] = pack2(2 * j < valid ? h.x : 0.0f, 2 * j + 1 < valid ? h.y : 0.0f);
    }
  }
  uint32_t mag = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const float2 h = split2(acc[j]);
    mag = max(mag, max(__float_as_uint(h.x) & 0x7FFFFFFFu, __float_as_uint(h.y) & 0x7FFFFFFFu));
  }
  finite = mag < 0x7F800000u;
  if (!finite) {
    mag = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const float2 h = split2(acc[j]);
      mag = max(mag, max(finite_mag_bits(h.x), finite_mag_bits(h.y)));
    }
  }
  return mag;
}

// columns 16 i .. 16 i + 15 of swiglu64's result in e4m3
__device__ __forceinline__ uint4 quant_columns(const uint64_t (&acc)[64], int i, float inv,
                                               bool finite) {
  float f[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 h = split2(acc[8 * i + j]);
    f[2 * j] = h.x;
    f[2 * j + 1] = h.y;
  }
  return finite ? quant16<true>(f, inv) : quant16<false>(f, inv);
}

}  // namespace gf
