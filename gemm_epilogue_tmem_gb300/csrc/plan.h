// The plan object behind include/gf.h, shared by the host entry points.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include <mutex>

#include "gf.h"

struct gf_plan {
  int64_t m, n, k;
  gf_dtype dtype;
  int epi;               // gf::Epi code (the public gf_epilog values, plus SwiGLU forms)
  gf_bias_axis bias_axis;
  gf_b_layout b_layout;
  int device;
  int num_sms;
  int tile_n;
  int forced_tile_n;
  int forced_kernel;     // 0 auto, 1 single CTA, 2 CTA pair, 3 CTA pair with 256 x 512 tiles
  int forced_group_m;    // 0 auto, else row (or column) blocks per raster group
  int forced_raster;     // 0 auto, 1 groups of row blocks, 2 groups of column blocks
  int raster_n;          // 1: raster groups of column blocks (B panels stay in L2)
  int l2_hint_a, l2_hint_b;  // L2 eviction policy of the A / B loads (0 none, 1 first, 2 last)
  int one_tile_per_cta;  // 1: grid of one tile per CTA (pair); the hardware orders the tiles
  int static_schedule;   // 1: persistent CTA pairs walk every gridDim-th tile (default: counter)
  int pair;              // the plan uses the CTA-pair kernel
  int wide;              // ... with 256 x 512 tiles
  int max_pair_clusters; // resident CTA pairs (0: the pair kernel cannot run)
  int stages;
  int grid;
  int num_m_blocks, num_n_blocks, num_k_blocks, num_tiles, group_m;
  gf_bgrad_mode bgrad_mode;
  uint64_t wait_limit_ns;
  int drop_load;
  int32_t* d_status;     // device status word (bounded-wait time-outs)
  float* d_partials;     // [num_m_blocks][n] fp32, DRELU_BGRAD two-pass only
  size_t partial_bytes;
  int forced_split;      // 0 the plan's choice, 1 no split, else k-splits per tile
  int split_from;        // CTA-pair split k: the first tile split into k-split units
  int k_splits;          // single-CTA kernel: CTAs sharing the k-blocks of one tile
  int kb_per_split;
  void* d_splitk;        // split-k partial sums, then the per-tile counters
  size_t splitk_bytes;   // capacity of d_splitk
  size_t splitk_cnt_offset;
  int pdl;               // 1: launches overlap their set-up with the previous kernel
  // Tensor maps of the last execute, reused while the operand pointers and
  // the plan's tiling are unchanged (encoding them is host work on every
  // call otherwise). `gen` counts tiling changes; the cache is valid for
  // cache_gen == gen.
  uint64_t gen;
  uint64_t cache_gen;
  bool cache_valid;
  const void* cache_A;
  const void* cache_B;
  const void* cache_B2;
  const void* cache_out;
  const void* cache_aux;
  bool cache_b_mn_3d;
  CUtensorMap cache_tmA, cache_tmB, cache_tmB2, cache_tmOut, cache_tmAux;
  std::mutex cache_mu;
  // gf_fp8_matmul_plan (m, n, k above): groups of rows with a B each
  int64_t groups;
  int kernel;            // 1, 2 narrow, 3 single CTA, 4 CTA pair
  int tile_rows;         // rows of a tile
  // gf_moe_plan: m = tokens, k = hidden
  int64_t topk, experts;
  int chunk_tokens;      // tokens per CTA of the sort
  int num_chunks;
  int fused;             // little to copy: the sort kernel does that too
  void* d_work;          // e4m3 products: counters and partial sums of split tiles
  size_t work_bytes;
};
