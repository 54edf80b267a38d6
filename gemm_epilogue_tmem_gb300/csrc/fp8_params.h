// Parameter block and launchers of the block-scaled e4m3 products.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gf {

constexpr int kFp8MaxGroups = 1024;

struct Fp8Params {
  int32_t M, N;             // rows of all groups, columns of one B
  int32_t groups;
  int32_t num_k_blocks;     // blocks of 128
  int32_t num_n_blocks;     // scale blocks of 128 columns
  const int32_t* offsets;   // [groups + 1], NULL: one group of all rows
  const float* a_scale;     // [M][num_k_blocks]
  const float* b_scale;     // [groups][num_n_blocks][num_k_blocks]
  const float* b2_scale;
  void* out;                // 16-bit [M][N], or e4m3 bytes
  float* out_scale;         // [M][num_n_blocks]
  // narrow kernel: partial sums of the tiles that several CTAs share, two
  // slots per CTA, and a counter per CTA (zero between launches)
  float* partials;
  int32_t* counters;
  int32_t* status;
  uint64_t wait_limit_ns;
  int32_t drop_load;        // test hook: 1-based index of a stage load to skip (0: none)
};

struct Fp8LaunchArgs {
  const CUtensorMap* tmA;   // the rows
  const CUtensorMap* tmB;   // B, and B2 (else = tmB)
  const CUtensorMap* tmB2;
  const Fp8Params* params;
  int grid;
  int bf16;
  int dual;                 // SwiGLU: two products, e4m3 out
  int tile_rows;            // rows of a tile of the narrow kernel
  int pdl;
  cudaStream_t stream;
};

// What it costs the narrow kernel to join the parts of split tiles, in k-blocks
// of a CTA's time (3 to 6 us)
__host__ __device__ constexpr int fp8_join_blocks(int tile_rows, int dual) {
  return dual ? 12 : tile_rows == 16 ? 15 : 20;
}
// The share of a grid's rounds, in percent, from which on it takes tiles whole
__host__ __device__ constexpr int fp8_whole_fill(int64_t rounds) { return rounds > 1 ? 65 : 60; }

// The CTAs over which the narrow kernel splits `tiles` tiles of kb k-blocks, each CTA
// having some k-blocks of them laid end to end; 0: it takes the tiles whole. They
// have at least four k-blocks each, and every tile the same number of CTAs where
// there are two or more for each, so that none has parts of two to join (1 x 4096 x
// 8192 10.7 us, otherwise 12.3).
__host__ __device__ inline int fp8_split_ctas(int tiles, int kb, int grid, int tile_rows,
                                              int dual) {
  const int rounds = (tiles + grid - 1) / grid;
  const int64_t room = static_cast<int64_t>(rounds) * grid;
  if (100ll * tiles >= fp8_whole_fill(rounds) * room ||
      (room - tiles) * kb <= static_cast<int64_t>(fp8_join_blocks(tile_rows, dual)) * grid)
    return 0;
  const int64_t most = static_cast<int64_t>(tiles) * kb / 4;
  int ctas = most < 1 ? 1 : most < grid ? static_cast<int>(most) : grid;
  if (ctas >= 2 * static_cast<int64_t>(tiles)) ctas -= ctas % tiles;
  return ctas;
}
// The CTA c of them that has k-block `unit`, of `units` in all: c's are
// [units c / ctas, units (c + 1) / ctas).
__host__ __device__ inline int fp8_unit_owner(int64_t unit, int64_t units, int ctas) {
  return static_cast<int>(((unit + 1) * ctas - 1) / units);
}

// the narrow kernel: 128 columns of B x tile_rows (16 or 64) rows per tile
cudaError_t launch_fp8_narrow(const Fp8LaunchArgs& a);
int fp8_narrow_stages(int tile_rows, int dual);
size_t fp8_narrow_partial_bytes(int tile_rows, int dual, int grid);
// the single-CTA kernel: 128 rows x 256 columns (SwiGLU: 128) per tile
cudaError_t launch_fp8_single(const Fp8LaunchArgs& a);
int fp8_single_stages();
// the CTA-pair kernel: 256 rows x 256 columns (SwiGLU: 128) per tile
cudaError_t launch_fp8_wide(const Fp8LaunchArgs& a);
int fp8_wide_stages();
// resident CTA pairs (0 if the kernel cannot launch)
int fp8_wide_max_clusters();

}  // namespace gf
