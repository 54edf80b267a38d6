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

__device__ __forceinline__ float silu_mul(float g, float u) {
  // e^-g overflows to infinity below -88, where g / infinity is the limit 0
  return __fdividef(g, 1.0f + __expf(-g)) * u;
}

}  // namespace gf
