// Block-scaled e4m3 product on single CTAs, for groups of some ten to some
// hundred rows: a tile is 128 rows x 256 columns of B (SwiGLU: 128 columns of
// each of the two weights). With up to 128 rows a group every weight passes
// through one SM once; with more, a group leaves half as much of its last tile
// empty as it does in tiles of a CTA pair.
//
// The rows are the tensor core's 128-row side whatever their number: an
// instruction of 128 x N x 32 takes 128 cycles for every N up to 256 (measured,
// the rate at which that side's operand is read), so that 256 columns of B per
// instruction stream the weights through an SM at 64 bytes a cycle, above its
// share of the HBM rate.
//
// The tensor core sums one block of 128 along k into one of two 256-column
// accumulators in tensor memory; eight epilogue warps, two per 32 rows, add it
// times its two scales to fp32 sums in registers (lane = row). The scales come
// through a ring in shared memory that a warp of its own fills, kScaleGroup blocks
// at a time (one at a time, that warp held up the epilogue's: 168 against 137 us, 64
// groups of 192 rows, 4096 x 2048). Warps without rows in a tile release its
// accumulators unread.
//
// What bounds it: with few rows HBM (64 groups of 32 or 64 rows, 0.54 GB of
// weights: 87-90 us, 90 % of the copy rate); with 128 rows and more shared
// memory, through which the 48 KB of a k-block pass twice, written by the loads and
// read by the tensor core, in 768 cycles at 128 bytes a cycle (64 groups of 128 rows
// 112 us, of 512 290-310; the CTA pair, which brings 32 KB for the same products
// of each SM, 133 and 306-323).
//
// Roles: warpgroup 0 = TMA producer, MMA issue, scale loads, one idle warp;
// warpgroups 1 and 2 epilogue. All waits are bounded.
#include "fp8_common.cuh"

namespace gf {
namespace {

constexpr int kThreadsSingle = 384;
constexpr int kCtlWarps = 4;
// registers per thread at launch (65536 / 384, in steps of 8), and after the
// redistribution from the control to the epilogue warpgroups
constexpr int kLaunchRegs = 168, kCtlRegs = 56, kEpiRegs = 224;
static_assert(128 * kCtlRegs + 256 * kEpiRegs <= kThreadsSingle * kLaunchRegs,
              "register redistribution within the launch's registers");
constexpr int kBPart = 128 * 128;  // 128 rows of a weight
constexpr int kScaleGroup = 8;     // blocks whose scales come together
constexpr int kRing = 2;           // such groups in flight
constexpr int kPad = 144;          // staged row: 128 bytes + 16 against bank conflicts

constexpr int TR = 128;            // rows of a tile
constexpr int kStageBytes = 3 * kBPart;
constexpr int kEpiWarps = 8;
constexpr int kEpiThreads = 32 * kEpiWarps;
constexpr int kStaging = kEpiWarps * 32 * kPad;
constexpr int kSlot = TR + 4;      // floats of a ring slot: rows, two column blocks
constexpr int kTable = 2 * (kFp8MaxGroups + 2) * 4;
constexpr int kFixed = kSmemAlignSlack + kSmemCtrlBytes + kStaging +
                       kRing * kScaleGroup * kSlot * 4 + 2 * TR * 4 + kTable;
constexpr int S = (kSmemPerCta - kFixed) / kStageBytes;
constexpr int kSmemSingle = kFixed + S * kStageBytes;
static_assert(S >= 3, "shared memory budget");
static_assert(16 * S + 48 + 16 * kRing <= kSmemCtrlBytes, "control region");

template <typename T, bool DUAL>
__global__ void __launch_bounds__(kThreadsSingle, 1)
    fp8_single_kernel(const __grid_constant__ CUtensorMap tmA,
                      const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmB2, const Fp8Params p) {
  constexpr int BN = DUAL ? 128 : 256;  // output columns of a tile
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t ctrl = base + S * kStageBytes;
  uint8_t* gctrl = smem_raw + (ctrl - raw);
  const uint32_t full0 = ctrl, empty0 = ctrl + 8u * S;
  const uint32_t tfull0 = ctrl + 16u * S, tempty0 = tfull0 + 16u;
  const uint32_t done_bar = tempty0 + 16u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gctrl + 16 * S + 40);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gctrl + 16 * S + 44);
  const uint32_t sfull0 = ctrl + 16u * S + 48u, sempty0 = sfull0 + 8u * kRing;
  uint8_t* staging = gctrl + kSmemCtrlBytes;
  float* ring = reinterpret_cast<float*>(staging + kStaging);
  uint32_t* row_mag = reinterpret_cast<uint32_t*>(ring + kRing * kScaleGroup * kSlot);
  GroupTable table;
  table.row0 = reinterpret_cast<int32_t*>(row_mag + 2 * TR);
  table.tile0 = table.row0 + kFp8MaxGroups + 2;

  const int warp = threadIdx.x >> 5;
  const uint32_t lane = lane_id();
  const int KB = p.num_k_blocks;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8u * s, 1);
      mbar_init(empty0 + 8u * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8u * b, 1);
      mbar_init(tempty0 + 8u * b, kEpiWarps);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(sfull0 + 8u * i, 32);
      mbar_init(sempty0 + 8u * i, kEpiWarps);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    if (KB > 0) {
      prefetch_tmap(&tmA);
      prefetch_tmap(&tmB);
      if (DUAL) prefetch_tmap(&tmB2);
    }
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  grid_dep_wait();
  grid_dep_launch();
  const int col_tiles = (p.N + BN - 1) / BN;
  build_group_table(p, table, TR, col_tiles);
  const int num_tiles = table.tile0[p.groups + 1];
  const int product_tiles = KB > 0 ? table.tile0[p.groups] : 0;  // the others are zeros
  bool aborted = false;

  const int cta = static_cast<int>(blockIdx.x), grid = static_cast<int>(gridDim.x);

  // tile t: its group, first row, rows and column tile
  auto tile_at = [&](int t, int& g, int& row, int& rows, int& nt) {
    g = group_of_tile(table, p.groups, t);
    const int first = table.row0[g], last = table.row0[g + 1];
    const int row_tiles = (last - first + TR - 1) / TR;
    const int i = t - table.tile0[g];
    nt = i / row_tiles;  // the row tiles of one B panel follow each other: it stays in L2
    row = first + (i - nt * row_tiles) * TR;
    rows = min(TR, last - row);
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
      for (int t = cta; t < product_tiles && ok; t += grid) {
        int g, row, rows, nt;
        tile_at(t, g, row, rows, nt);
        const int b_row = g * p.N + nt * BN;
        for (int kb = 0; kb < KB; ++kb) {
          ok = mbar_wait_bounded(empty0 + 8u * stage, phase ^ 1u, abort_flag, p.wait_limit_ns);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) {
            fp8_raise(p, abort_flag, ST_TIMEOUT_PRODUCER);
            aborted = true;
            break;
          }
          ++loads;
          if (loads != p.drop_load) {
            const uint32_t fb = full0 + 8u * stage;
            const uint32_t dst = base + stage * kStageBytes;
            if (e) mbar_arrive_expect_tx(fb, kStageBytes);
            __syncwarp();
            tma_load_f8<false>(dst, &tmB, fb, kb * 128, b_row, e);
            // the other 128 columns (past the matrix the box is zeros), or up's
            tma_load_f8<false>(dst + kBPart, DUAL ? &tmB2 : &tmB, fb, kb * 128,
                               DUAL ? b_row : b_row + 128, e);
            tma_load_f8<false>(dst + 2 * kBPart, &tmA, fb, kb * 128, row, e);
            issued |= 1u << stage;
            issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          }
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      for (int s = 0; s < S; ++s)
        if ((issued >> s & 1u) && !mbar_wait_bounded(full0 + 8u * s, issued_phase >> s & 1u,
                                                     nullptr, p.wait_limit_ns))
          fp8_raise(p, abort_flag, ST_TIMEOUT_DRAIN);
      __syncwarp();
    } else if (warp == 1) {
      // --------------------------------------------------------------- MMA
      constexpr uint32_t idesc = idesc_e4m3(128, 256);
      const uint32_t e = elect_one();
      const uint64_t desc0 = sdesc_sw128(base, 16, 1024);
      int stage = 0, buf = 0;
      uint32_t phase = 0, bphase = 0;
      bool ok = true;
      const int tiles = product_tiles > cta ? (product_tiles - cta - 1) / grid + 1 : 0;
      for (int64_t i = static_cast<int64_t>(tiles) * KB; i > 0; --i) {
        ok = mbar_wait_bounded(full0 + 8u * stage, phase, abort_flag, p.wait_limit_ns);
        if (!__all_sync(0xFFFFFFFFu, ok)) {
          fp8_raise(p, abort_flag, ST_TIMEOUT_MMA_SMEM);
          aborted = true;
          break;
        }
        ok = mbar_wait_bounded(tempty0 + 8u * buf, bphase ^ 1u, abort_flag, p.wait_limit_ns);
        if (!__all_sync(0xFFFFFFFFu, ok)) {
          fp8_raise(p, abort_flag, ST_TIMEOUT_MMA_TMEM);
          aborted = true;
          break;
        }
        tc_fence_after();
        // (a descriptor's address field counts 16 bytes)
        const uint64_t bdesc = desc0 + static_cast<uint64_t>(stage * (kStageBytes / 16));
        const uint64_t adesc = bdesc + 2 * kBPart / 16;
        const uint32_t d = tmem_base + 256u * static_cast<uint32_t>(buf);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_f8<false>(d, adesc + 2 * kk, bdesc + 2 * kk, idesc, kk != 0, e);
        umma_commit_f8<false>(empty0 + 8u * stage, e);
        umma_commit_f8<false>(tfull0 + 8u * buf, e);
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
        buf ^= 1;
        bphase ^= buf == 0 ? 1u : 0u;
      }
      umma_commit_f8<false>(done_bar, e);
      if (!mbar_wait_bounded(done_bar, 0, nullptr, p.wait_limit_ns))
        fp8_raise(p, abort_flag, ST_TIMEOUT_DRAIN);
      __syncwarp();
    } else if (warp == 2) {
      // ------------------------------------------------------- scale loads
      int slot = 0;
      uint32_t phase = 0;
      bool ok = true;
      const uint32_t ring_s = smem_u32(ring);
      for (int t = cta; t < product_tiles && ok; t += grid) {
        int g, row, rows, nt;
        tile_at(t, g, row, rows, nt);
        const float* as = p.a_scale + static_cast<int64_t>(row + static_cast<int>(lane)) * KB;
        // lanes 0 and 1: the scales of the tile's two column blocks (SwiGLU:
        // of one block of each weight)
        const int nb = DUAL ? nt : 2 * nt + static_cast<int>(lane & 1u);
        const float* bs = (DUAL && lane == 1 ? p.b2_scale : p.b_scale) +
                          (static_cast<int64_t>(g) * p.num_n_blocks + nb) * KB;
        const bool b_in = lane < 2 && nb < p.num_n_blocks;
        for (int kb0 = 0; kb0 < KB; kb0 += kScaleGroup) {
          ok = mbar_wait_bounded(sempty0 + 8u * slot, phase ^ 1u, abort_flag, p.wait_limit_ns);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) {
            fp8_raise(p, abort_flag, ST_TIMEOUT_PRODUCER);
            aborted = true;
            break;
          }
          const int last = min(kb0 + kScaleGroup, KB);
          uint32_t dst = ring_s + 4u * (kSlot * kScaleGroup * slot + lane);
          for (int kb = kb0; kb < last; ++kb, dst += 4u * kSlot) {
#pragma unroll
            for (int i = 0; i < TR / 32; ++i) {
              const bool in = 32 * i + static_cast<int>(lane) < rows;
              cp_async_4(dst + 128u * i,
                         in ? as + static_cast<int64_t>(32 * i) * KB + kb : p.a_scale, in);
            }
            if (lane < 2) cp_async_4(dst + 4u * TR, b_in ? bs + kb : p.b_scale, b_in);
          }
          cp_async_arrive(sfull0 + 8u * slot);
          if (++slot == kRing) {
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
    const int r = 32 * q + static_cast<int>(lane);  // this thread's row of a tile
    const uint32_t col_a = DUAL ? 64u * sub : 128u * sub;
    const uint32_t col_b = DUAL ? 128u + 64u * sub : 128u * sub + 64u;
    uint8_t* stg = staging + (q * 2 + sub) * 32 * kPad;
    int buf = 0, slot = 0;
    uint32_t bphase = 0, sphase = 0;
    uint64_t acc[64];

    auto store_tile = [&](int row, int rows, int nt) {
      const bool busy = 32 * q < rows;
      if constexpr (!DUAL) {
        if (!busy) return;
        // 64 columns at a time through shared memory: 128-byte row segments
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 f = split2(acc[32 * half + 4 * j + i]);
              w[i] = Pair16<T>::pack(f.x, f.y);
            }
            *reinterpret_cast<uint4*>(stg + lane * kPad + 16 * j) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
          __syncwarp();
          const int n = nt * 256 + 128 * sub + 64 * half + 8 * static_cast<int>(lane & 7u);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int rr = 4 * j + static_cast<int>(lane >> 3);
            const uint4 w = *reinterpret_cast<const uint4*>(stg + rr * kPad + 16 * (lane & 7u));
            if (32 * q + rr < rows && n < p.N)
              *reinterpret_cast<uint4*>(static_cast<T*>(p.out) +
                                        static_cast<int64_t>(row + 32 * q + rr) * p.N + n) = w;
          }
        }
      } else {
        // h of this row's 64 columns, its largest magnitude over the tile's
        // 128 with the other warp of the quarter
        const int n0 = nt * 128 + 64 * sub;
        bool finite = true;
        uint32_t mag = 0;
        if (busy) {
          mag = swiglu64(acc, p.N - n0, finite);
          row_mag[TR * sub + r] = mag;
        }
        named_bar_sync(1, kEpiThreads);
        if (busy) {
          mag = max(mag, row_mag[TR * (sub ^ 1) + r]);
          float inv;
          const float sc = e4m3_scale(mag, inv);
          if (sub == 0 && r < rows)
            p.out_scale[static_cast<int64_t>(row + r) * p.num_n_blocks + nt] = sc;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(stg + lane * 80 + 16 * j) =
                quant_columns(acc, j, inv, finite);
          __syncwarp();
          const int n = n0 + 16 * static_cast<int>(lane & 3u);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int rr = 8 * j + static_cast<int>(lane >> 2);
            const uint4 w = *reinterpret_cast<const uint4*>(stg + rr * 80 + 16 * (lane & 3u));
            if (32 * q + rr < rows && n < p.N)
              *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) +
                                        static_cast<int64_t>(row + 32 * q + rr) * p.N + n) = w;
          }
        }
        // the magnitudes and the staging are read before the next tile
        named_bar_sync(1, kEpiThreads);
      }
    };

    bool ok = true;
    for (int t = cta; t < product_tiles; t += grid) {
      int g, row, rows, nt;
      tile_at(t, g, row, rows, nt);
      const bool busy = 32 * q < rows;  // the warp has rows of this tile
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = 0ull;
      for (int left = KB; left > 0 && ok; left -= kScaleGroup) {
        ok = mbar_wait_bounded(sfull0 + 8u * slot, sphase, abort_flag, p.wait_limit_ns);
        const float* sc = ring + kSlot * kScaleGroup * slot;
        for (int kb = min(left, kScaleGroup); kb > 0; --kb, sc += kSlot) {
          const float sa = sc[r];
          const uint64_t s_a = both(sa * sc[DUAL ? TR : TR + sub]);
          const uint64_t s_b = DUAL ? both(sa * sc[TR + 1]) : s_a;
          ok = mbar_wait_bounded(tfull0 + 8u * buf, bphase, abort_flag, p.wait_limit_ns) && ok;
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint32_t taddr = tmem_base + (static_cast<uint32_t>(32 * q) << 16) +
                                 256u * static_cast<uint32_t>(buf);
          if (busy) {
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
                if (lane == 0) mbar_arrive(tempty0 + 8u * buf);
              }
#pragma unroll
              for (int j = 0; j < 32; ++j)
                fma2(acc[32 * c + j], v[j >> 4][2 * (j & 15)], v[j >> 4][2 * (j & 15) + 1],
                     c == 0 ? s_a : s_b);
            }
          } else {
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty0 + 8u * buf);
          }
          buf ^= 1;
          bphase ^= buf == 0 ? 1u : 0u;
        }
        __syncwarp();  // all lanes have read their scales
        if (lane == 0) mbar_arrive(sempty0 + 8u * slot);
        if (++slot == kRing) {
          slot = 0;
          sphase ^= 1u;
        }
      }
      // all epilogue warps agree on the outcome (barriers follow)
      ok = !named_bar_red_or(1, kEpiThreads, !ok);
      if (!ok) {
        fp8_raise(p, abort_flag, ST_TIMEOUT_EPILOGUE);
        aborted = true;
        break;
      }
      store_tile(row, rows, nt);
    }
    // the rows of no group (and every row of a product over nothing)
    if (ok) {
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = 0ull;
      for (int t = product_tiles + cta; t < num_tiles; t += grid) {
        int g, row, rows, nt;
        tile_at(t, g, row, rows, nt);
        store_tile(row, rows, nt);
      }
    }
  }

  // a CTA that gave up may still have loads in flight towards its shared memory
  if (__syncthreads_or(aborted ? 1 : 0) || *abort_flag) sleep_ns(200000);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

template <typename T, bool DUAL>
cudaError_t launch_single(const Fp8LaunchArgs& a) {
  auto kernel = fp8_single_kernel<T, DUAL>;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemSingle);
  if (e != cudaSuccess) return e;
  // the redistribution of registers adds up only for this launch register
  // count: refuse to launch a build that differs
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, kernel);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidKernelImage;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.grid, 1, 1);
  cfg.blockDim = dim3(kThreadsSingle, 1, 1);
  cfg.dynamicSmemBytes = kSmemSingle;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = a.pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, *a.tmA, *a.tmB, *a.tmB2, *a.params);
}

}  // namespace

int fp8_single_stages() { return S; }

cudaError_t launch_fp8_single(const Fp8LaunchArgs& a) {
  if (a.dual) return launch_single<__half, true>(a);
  return a.bf16 ? launch_single<__nv_bfloat16, false>(a) : launch_single<__half, false>(a);
}

}  // namespace gf
