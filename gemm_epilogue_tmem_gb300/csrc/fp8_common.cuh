// What the block-scaled e4m3 kernels share: the table of groups and tiles,
// the tensor-core instruction and its descriptor, error reporting.
#pragma once

#include <type_traits>

#include "fp8.cuh"
#include "fp8_params.h"
#include "params.h"
#include "ptx.cuh"

namespace gf {

// D[tmem] (+)= A[smem desc] x B[smem desc], kind::f8f6f4 (8-bit in, fp32 acc).
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor, kind::f8f6f4: D fp32, A and B e4m3 (format 0), both
// K-major, N >> 3 at [17,23), M >> 4 at [24,29).
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

// 32 lanes x 16 columns of 32-bit: thread t gets lane (base lane + t)
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld_wait_tied(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

__device__ __forceinline__ void fp8_raise(const Fp8Params& p, volatile int* abort_flag,
                                          int code) {
  *abort_flag = 1;
  atomicOr(p.status, code);
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
