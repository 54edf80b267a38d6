// Block-scaled e4m3 product for many rows a group: a cluster of two CTAs
// computes 256 rows x 256 columns of B with tcgen05.mma.cta_group::2 (for the
// SwiGLU form 128 columns of each of the two weights, side by side).
//
// The tensor core sums one block of 128 along k (one 128-byte-swizzled stage of
// 32 KB per CTA, four K = 32 instructions) into one of two 256-column
// accumulators in tensor memory. Eight epilogue warps per CTA, two per lane
// quarter, add it, times its two scales, to the tile's fp32 sums, which stay in
// registers (128 rows x 256 columns per CTA, 128 registers a thread): lane =
// row, so that the product of the two scales is one number per thread and
// block, and the addition two columns per instruction. The registers hold no
// more columns than these, which bounds the tile.
//
// What bounds it: an accumulator's way round. A block's products take 512
// cycles; its commit, the epilogue's wake-up, loads and release and the next
// issue take about 900 more, of which the second accumulator hides its own
// 512: 713 cycles a block (0.375 us, from k = 1024 against k = 4096). Tensor
// memory has no room for a third accumulator of this width, and with four of 128
// columns the N = 128 instructions (365 cycles a half) are the slower choice.
// Measured at m = 8192, n = 16384, k = 4096: 378 us, 2.9 PFLOP/s; 419-436 us in a
// steady loop at the power cap.
//
// The rows' scales lie a row apart in memory, so that a warp's load of one block
// touches 32 sectors: a warp of its own copies them asynchronously into a ring
// in shared memory, ahead of the epilogue, kScaleGroup blocks at a time. With one
// block at a time, released with the accumulator, that warp woke up and loaded
// exactly when the epilogue warps of its scheduler were in the accumulator's
// way: 420 us instead of 383.
//
// A finished tile goes through a shared-memory staging buffer of each warp's own
// and leaves it in whole row segments (by one bulk copy a row instead, which
// a warp issues one after the other: 527 against 503 us, 64 groups of 512 rows,
// gate and up projections of 4096 x 2048).
//
// Roles: warpgroup 0 = TMA producer, MMA issue (leader CTA), scale loads, one
// idle warp; warpgroups 1 and 2 epilogue. All waits are bounded.
#include "fp8_common.cuh"

namespace gf {
namespace {

constexpr int kThreadsWide = 384;
constexpr int kCtlWarps = 4;
constexpr int kEpiWarps = 8;
// registers per thread at launch (65536 / 384, in steps of 8), and after the
// redistribution from the control to the epilogue warpgroups
constexpr int kLaunchRegs = 168, kCtlRegs = 56, kEpiRegs = 224;
static_assert(128 * kCtlRegs + 256 * kEpiRegs <= kThreadsWide * kLaunchRegs,
              "register redistribution within the launch's registers");
constexpr int kPartBytes = 128 * 128;            // 128 rows of one operand
constexpr int kStageBytes = 2 * kPartBytes;      // per CTA
// staged row segment of a warp: 128 16-bit columns (SwiGLU: 64 bytes), and 16
// bytes against bank conflicts
constexpr int kStagePad = 272;
constexpr int kStagePadDual = 80;
constexpr int kStagingBytes = kEpiWarps * 32 * kStagePad;
constexpr int kScaleGroup = 8;                   // blocks whose scales come together
constexpr int kScaleRing = 2;                    // groups
constexpr int kScaleSlot = 132;                  // floats of a block: 128 rows, two column blocks
constexpr int kScaleBytes = kScaleRing * kScaleGroup * kScaleSlot * 4;
constexpr int kTableBytes = 2 * (kFp8MaxGroups + 2) * 4;
constexpr int kMagBytes = 2 * 128 * 4;
constexpr int kStagesWide = (kSmemPerCta - kSmemAlignSlack - kSmemCtrlBytes - kStagingBytes -
                             kTableBytes - kMagBytes - kScaleBytes) /
                            kStageBytes;
constexpr int kSmemWide = kSmemAlignSlack + kStagesWide * kStageBytes + kSmemCtrlBytes +
                          kStagingBytes + kTableBytes + kMagBytes + kScaleBytes;
// row tiles visited together, column by column: 442 us in a steady loop at
// m = 8192, n = 16384, k = 4096, against 448 with 8 and 458 with 4
constexpr int kRasterRows = 16;

template <typename T, bool DUAL>
__global__ void __launch_bounds__(kThreadsWide, 1)
    fp8_wide_kernel(const __grid_constant__ CUtensorMap tmA,
                    const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmB2, const Fp8Params p) {
  constexpr int S = kStagesWide;
  constexpr int BN = DUAL ? 128 : 256;  // output columns of a tile
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t ctrl = base + S * kStageBytes;
  uint8_t* gctrl = smem_raw + (ctrl - raw);
  const uint32_t full0 = ctrl;             // leader: stage filled (both CTAs' bytes)
  const uint32_t empty0 = ctrl + 8u * S;   // both: stage consumed
  const uint32_t tfull0 = ctrl + 16u * S;  // both: accumulator ready
  const uint32_t tempty0 = tfull0 + 16u;   // leader: accumulator read by both CTAs
  const uint32_t done_bar = tempty0 + 16u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gctrl + 16 * S + 40);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gctrl + 16 * S + 44);
  const uint32_t sfull0 = ctrl + 16u * S + 48u;       // scales of a block ready
  const uint32_t sempty0 = sfull0 + 8u * kScaleRing;  // ... read by the epilogue warps
  static_assert(16 * S + 48 + 16 * kScaleRing <= kSmemCtrlBytes, "control region");
  uint8_t* staging = gctrl + kSmemCtrlBytes;
  GroupTable table;
  table.row0 = reinterpret_cast<int32_t*>(staging + kStagingBytes);
  table.tile0 = table.row0 + kFp8MaxGroups + 2;
  uint32_t* row_mag = reinterpret_cast<uint32_t*>(staging + kStagingBytes + kTableBytes);
  float* scales = reinterpret_cast<float*>(staging + kStagingBytes + kTableBytes + kMagBytes);

  const int warp = threadIdx.x >> 5;
  const uint32_t lane = lane_id();
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster_id = blockIdx.x >> 1;
  const int num_clusters = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8u * s, 1);
      mbar_init(empty0 + 8u * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8u * b, 1);
      mbar_init(tempty0 + 8u * b, 2 * kEpiWarps);
    }
    mbar_init(done_bar, 1);
    for (int i = 0; i < kScaleRing; ++i) {
      mbar_init(sfull0 + 8u * i, 32);
      mbar_init(sempty0 + 8u * i, kEpiWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
    if (p.num_k_blocks > 0) {
      prefetch_tmap(&tmA);
      prefetch_tmap(&tmB);
      if (DUAL) prefetch_tmap(&tmB2);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();  // barriers of both CTAs initialised before any remote use
  tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  grid_dep_wait();
  grid_dep_launch();
  const int col_tiles = (p.N + BN - 1) / BN;
  build_group_table(p, table, 256, col_tiles);
  const int num_tiles = table.tile0[p.groups + 1];
  const int KB = p.num_k_blocks;
  bool aborted = false;

  // tile t: its group, first row (of the pair), end of the group's rows,
  // column tile; row tiles in runs of kRasterRows, so that the tiles in
  // flight share their operand panels in L2
  auto tile_at = [&](int t, int& g, int& row, int& row_end, int& nt) {
    g = group_of_tile(table, p.groups, t);
    const int first = table.row0[g];
    row_end = table.row0[g + 1];
    const int row_tiles = (row_end - first + 255) / 256;
    int i = t - table.tile0[g];
    const int run = i / (kRasterRows * col_tiles);
    i -= run * kRasterRows * col_tiles;
    const int rows = min(kRasterRows, row_tiles - run * kRasterRows);
    nt = i / rows;
    row = first + (run * kRasterRows + i - nt * rows) * 256;
  };

  if (warp < kCtlWarps) {
    setmaxnreg_dec<kCtlRegs>();
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      const uint32_t e = elect_one();
      int stage = 0;
      uint32_t phase = 0;
      int loads = 0;
      bool ok = true;
      uint32_t issued = 0, issued_phase = 0;  // bit s: a load of stage s, and its phase
      const uint32_t leader_full = mapa_shared(full0, 0);
      for (int t = cluster_id; t < num_tiles && ok; t += num_clusters) {
        int g, row, row_end, nt;
        tile_at(t, g, row, row_end, nt);
        const int nkb = g < p.groups ? KB : 0;
        const int a_row = row + 128 * static_cast<int>(rank);
        const int b_row = g * p.N + (DUAL ? nt * 128 : nt * 256 + 128 * static_cast<int>(rank));
        const CUtensorMap* mb = DUAL && rank == 1 ? &tmB2 : &tmB;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(empty0 + 8u * stage, phase ^ 1u,
                                                         abort_flag, p.wait_limit_ns))) {
            fp8_raise(p, abort_flag, ST_TIMEOUT_PRODUCER);
            aborted = true;
            ok = false;
            break;
          }
          ++loads;
          if (loads != p.drop_load) {
            const uint32_t fb = leader_full + 8u * stage;
            const uint32_t dst = base + stage * kStageBytes;
            if (leader && e) mbar_arrive_expect_tx(full0 + 8u * stage, 2u * kStageBytes);
            __syncwarp();
            tma_load_f8<true>(dst, &tmA, fb, kb * 128, a_row, e);
            tma_load_f8<true>(dst + kPartBytes, mb, fb, kb * 128, b_row, e);
            issued |= 1u << stage;
            issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          }
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // the leader's full barriers count both CTAs' bytes: when they have
      // completed, every load of the pair has landed
      if (leader)
        for (int s = 0; s < S; ++s)
          if ((issued >> s & 1u) && !mbar_wait_bounded(full0 + 8u * s, issued_phase >> s & 1u,
                                                       nullptr, p.wait_limit_ns))
            fp8_raise(p, abort_flag, ST_TIMEOUT_DRAIN);
      __syncwarp();
    } else if (warp == 1) {
      // ----------------------------------------------------- MMA (leader)
      if (leader) {
        constexpr uint32_t idesc = idesc_e4m3(256, 256);
        const uint32_t e = elect_one();
        const uint64_t desc0 = sdesc_sw128(base, 16, 1024);
        int stage = 0, buf = 0;
        uint32_t phase = 0, bphase = 0;
        bool ok = true;
        // all tiles of products have KB blocks
        const int tiles = table.tile0[p.groups];
        const int mine = tiles > cluster_id ? (tiles - cluster_id - 1) / num_clusters + 1 : 0;
        for (int64_t i = static_cast<int64_t>(mine) * KB; i > 0; --i) {
          ok = mbar_wait_bounded(full0 + 8u * stage, phase, abort_flag, p.wait_limit_ns);
          if (!__all_sync(0xFFFFFFFFu, ok)) {
            fp8_raise(p, abort_flag, ST_TIMEOUT_MMA_SMEM);
            aborted = true;
            break;
          }
          // the accumulator last: its release is what the pace hangs on
          ok = mbar_wait_bounded_cluster(tempty0 + 8u * buf, bphase ^ 1u, abort_flag,
                                         p.wait_limit_ns);
          if (!__all_sync(0xFFFFFFFFu, ok)) {
            fp8_raise(p, abort_flag, ST_TIMEOUT_MMA_TMEM);
            aborted = true;
            break;
          }
          tc_fence_after();
          // (a descriptor's address field counts 16 bytes)
          const uint64_t adesc = desc0 + static_cast<uint64_t>(stage * (kStageBytes / 16));
          const uint64_t bdesc = adesc + kPartBytes / 16;
          const uint32_t d = tmem_base + 256u * static_cast<uint32_t>(buf);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_f8<true>(d, adesc + 2 * kk, bdesc + 2 * kk, idesc, kk != 0, e);
          umma_commit_f8<true>(empty0 + 8u * stage, e);
          umma_commit_f8<true>(tfull0 + 8u * buf, e);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
          buf ^= 1;
          bphase ^= buf == 0 ? 1u : 0u;
        }
        if (e) umma_commit_pair(done_bar, 0x1);
        if (!mbar_wait_bounded(done_bar, 0, nullptr, p.wait_limit_ns))
          fp8_raise(p, abort_flag, ST_TIMEOUT_DRAIN);
      }
      __syncwarp();
    } else if (warp == 2) {
      // ------------------------------------------------------- scale loads
      int slot = 0;
      uint32_t phase = 0;
      bool ok = true;
      const uint32_t ring = smem_u32(scales);
      for (int t = cluster_id; t < num_tiles && ok; t += num_clusters) {
        int g, row, row_end, nt;
        tile_at(t, g, row, row_end, nt);
        const int nkb = g < p.groups ? KB : 0;
        const int r0 = row + 128 * static_cast<int>(rank) + static_cast<int>(lane);
        const float* as = p.a_scale + static_cast<int64_t>(r0) * KB;
        // lanes 0 and 1: the scales of the tile's two column blocks (SwiGLU:
        // of one block of each weight)
        const int nb = DUAL ? nt : 2 * nt + static_cast<int>(lane & 1u);
        const float* bs = (DUAL && lane == 1 ? p.b2_scale : p.b_scale) +
                          (static_cast<int64_t>(g) * p.num_n_blocks + nb) * KB;
        const bool b_in = lane < 2 && nb < p.num_n_blocks;
        for (int kb0 = 0; kb0 < nkb; kb0 += kScaleGroup) {
          ok = mbar_wait_bounded(sempty0 + 8u * slot, phase ^ 1u, abort_flag, p.wait_limit_ns);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) {
            fp8_raise(p, abort_flag, ST_TIMEOUT_PRODUCER);
            aborted = true;
            break;
          }
          const int last = min(kb0 + kScaleGroup, nkb);
          uint32_t dst = ring + 4u * (kScaleSlot * kScaleGroup * slot + lane);
          for (int kb = kb0; kb < last; ++kb, dst += 4u * kScaleSlot) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool in = r0 + 32 * i < p.M;
              cp_async_4(dst + 128u * i,
                         in ? as + static_cast<int64_t>(32 * i) * KB + kb : p.a_scale, in);
            }
            if (lane < 2) cp_async_4(dst + 512u, b_in ? bs + kb : p.b_scale, b_in);
          }
          cp_async_arrive(sfull0 + 8u * slot);
          if (++slot == kScaleRing) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      cp_async_wait_all();  // no copy lands after the CTA is gone
    }
  } else {
    setmaxnreg_inc<kEpiRegs>();
    // -------------------------------------------------------------- epilogue
    const int ew = warp - kCtlWarps;
    const int q = warp & 3;   // tensor-memory lane quarter
    const int sub = ew >> 2;  // half of the columns (DUAL: of each weight's)
    const int row_in_tile = 128 * static_cast<int>(rank) + 32 * q + static_cast<int>(lane);
    const uint32_t tempty_leader = mapa_shared(tempty0, 0);
    // accumulator columns of this warp: two runs of 64
    const uint32_t col_a = DUAL ? 64u * sub : 128u * sub;
    const uint32_t col_b = DUAL ? 128u + 64u * sub : 128u * sub + 64u;
    constexpr int kPad = DUAL ? kStagePadDual : kStagePad;
    uint8_t* stg = staging + ew * 32 * kStagePad;  // this warp's rows
    uint8_t* my_stg = stg + lane * kPad;
    int buf = 0, slot = 0;
    uint32_t bphase = 0, sphase = 0;
    for (int t = cluster_id; t < num_tiles; t += num_clusters) {
      int g, row, row_end, nt;
      tile_at(t, g, row, row_end, nt);
      const int nkb = g < p.groups ? KB : 0;
      const int my_row = row + row_in_tile;
      uint64_t acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = 0ull;
      bool ok = true;
      for (int left = nkb; left > 0 && ok; left -= kScaleGroup) {
        ok = mbar_wait_bounded(sfull0 + 8u * slot, sphase, abort_flag, p.wait_limit_ns);
        const float* sc = scales + kScaleSlot * kScaleGroup * slot;
        for (int kb = min(left, kScaleGroup); kb > 0; --kb, sc += kScaleSlot) {
          const float sa = sc[32 * q + lane];
          const uint64_t s_a = both(sa * sc[DUAL ? 128 : 128 + sub]);
          const uint64_t s_b = DUAL ? both(sa * sc[129]) : s_a;
          ok = mbar_wait_bounded(tfull0 + 8u * buf, bphase, abort_flag, p.wait_limit_ns) && ok;
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint32_t taddr = tmem_base + (static_cast<uint32_t>(32 * q) << 16) +
                                 256u * static_cast<uint32_t>(buf);
          // 64 columns at a time: two loads in flight, and the accumulator is
          // released as soon as the second pair is in registers
          uint32_t v[2][32];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            tmem_ld_32x32b_x32(taddr + (c == 0 ? col_a : col_b), v[0]);
            tmem_ld_32x32b_x32(taddr + (c == 0 ? col_a : col_b) + 32u, v[1]);
            tmem_ld_wait_tied(v[0]);
            tmem_tie(v[1]);
            if (c == 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_remote_relaxed(tempty_leader + 8u * buf);
            }
#pragma unroll
            for (int j = 0; j < 32; ++j)
              fma2(acc[32 * c + j], v[j >> 4][2 * (j & 15)], v[j >> 4][2 * (j & 15) + 1],
                   c == 0 ? s_a : s_b);
          }
          buf ^= 1;
          bphase ^= buf == 0 ? 1u : 0u;
        }
        __syncwarp();  // all lanes have read their scales
        if (lane == 0) mbar_arrive(sempty0 + 8u * slot);
        if (++slot == kScaleRing) {
          slot = 0;
          sphase ^= 1u;
        }
      }
      // (DUAL: the two warps of a quarter agree on the outcome, a barrier follows)
      if constexpr (DUAL) ok = !named_bar_red_or(1 + q, 64, !ok);
      if (!ok) {
        fp8_raise(p, abort_flag, ST_TIMEOUT_EPILOGUE);
        aborted = true;
        break;
      }
      if constexpr (!DUAL) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = split2(acc[4 * j + i]);
            w[i] = Pair16<T>::pack(f.x, f.y);
          }
          *reinterpret_cast<uint4*>(my_stg + 16 * j) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
        const int n = nt * 256 + 128 * sub + 8 * static_cast<int>(lane & 15u);
        const int r0 = my_row - static_cast<int>(lane) + static_cast<int>(lane >> 4);
        T* dst = static_cast<T*>(p.out) + static_cast<int64_t>(r0) * p.N + n;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const uint4 w = *reinterpret_cast<const uint4*>(stg + (2 * j + (lane >> 4)) * kPad +
                                                          16 * (lane & 15u));
          if (r0 + 2 * j < row_end && n < p.N)
            *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(2 * j) * p.N) = w;
        }
        __syncwarp();
      } else {
        // h of this row's 64 columns, its largest magnitude over the tile's
        // 128 with the other warp of the quarter
        const int n = nt * 128 + 64 * sub;
        bool finite;
        uint32_t mag = swiglu64(acc, p.N - n, finite);
        row_mag[128 * sub + 32 * q + lane] = mag;
        named_bar_sync(1 + q, 64);
        mag = max(mag, row_mag[128 * (sub ^ 1) + 32 * q + lane]);
        float inv;
        const float sc = e4m3_scale(mag, inv);
        if (sub == 0 && my_row < row_end)
          p.out_scale[static_cast<int64_t>(my_row) * p.num_n_blocks + nt] = sc;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4*>(my_stg + 16 * j) = quant_columns(acc, j, inv, finite);
        __syncwarp();
        const int c0 = n + 16 * static_cast<int>(lane & 3u);
        const int r0 = my_row - static_cast<int>(lane) + static_cast<int>(lane >> 2);
        uint8_t* dst = static_cast<uint8_t*>(p.out) + static_cast<int64_t>(r0) * p.N + c0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 w = *reinterpret_cast<const uint4*>(stg + (8 * j + (lane >> 2)) * kPad +
                                                          16 * (lane & 3u));
          if (r0 + 8 * j < row_end && c0 < p.N)
            *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(8 * j) * p.N) = w;
        }
      }
    }
  }

  // a CTA that gave up may still have loads in flight towards its shared
  // memory that no barrier of its own tracks: give them time to land
  if (__syncthreads_or(aborted ? 1 : 0) || *abort_flag) sleep_ns(200000);
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

template <typename T, bool DUAL>
cudaError_t configure(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, const Fp8LaunchArgs& a) {
  auto kernel = fp8_wide_kernel<T, DUAL>;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemWide);
  if (e != cudaSuccess) return e;
  // the redistribution of registers adds up only for this launch register
  // count: refuse to launch a build that differs
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, kernel);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidKernelImage;
  cfg.gridDim = dim3(a.grid, 1, 1);
  cfg.blockDim = dim3(kThreadsWide, 1, 1);
  cfg.dynamicSmemBytes = kSmemWide;
  cfg.stream = a.stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = a.pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaSuccess;
}

template <typename T, bool DUAL>
cudaError_t launch_wide(const Fp8LaunchArgs& a) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  const cudaError_t e = configure<T, DUAL>(cfg, attr, a);
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, fp8_wide_kernel<T, DUAL>, *a.tmA, *a.tmB, *a.tmB2, *a.params);
}

}  // namespace

int fp8_wide_stages() { return kStagesWide; }

int fp8_wide_max_clusters() {
  Fp8LaunchArgs a = {};
  a.grid = 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  if (configure<__half, true>(cfg, attr, a) != cudaSuccess) return 0;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, fp8_wide_kernel<__half, true>, &cfg) != cudaSuccess)
    return 0;
  return n;
}

cudaError_t launch_fp8_wide(const Fp8LaunchArgs& a) {
  if (a.dual) return launch_wide<__half, true>(a);
  return a.bf16 ? launch_wide<__nv_bfloat16, false>(a) : launch_wide<__half, false>(a);
}

}  // namespace gf
