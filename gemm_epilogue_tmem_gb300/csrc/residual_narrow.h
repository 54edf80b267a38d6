// The product with a residual for few rows: its tiles and its launcher.
#pragma once

#include "launch.h"

namespace gf {

// rows of a tile: the least of 16, 32, 64 that holds the rows, 64 for more
__host__ __device__ constexpr int narrow_rows(int64_t m) { return m <= 16 ? 16 : m <= 32 ? 32 : 64; }

constexpr int kNarrowMaxSplits = 8;  // CTAs that share a tile: a cluster

int narrow_stages(int rows);
// The clusters of `splits` CTAs that can be resident at once, for tiles of `rows` rows.
int narrow_clusters(int rows, int splits);
// a.tile_n: rows of a tile; params->k_splits: CTAs a tile, a cluster
cudaError_t launch_residual_narrow(const LaunchArgs& a);

}  // namespace gf
