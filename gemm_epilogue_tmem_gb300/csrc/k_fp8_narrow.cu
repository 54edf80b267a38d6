// Block-scaled e4m3 product for few rows a group: a tile is 128 columns of B
// times TR rows, with B on the tensor core's 128-row side (D = B . A^T), so
// that a tile of 16 rows costs no more tensor work than 16 rows need and the
// whole CTA streams one operand, B, from HBM.
//
// The scales vary along k, so the tensor core sums one block of 128 at a time
// (one 128-byte-swizzled stage, four K = 32 instructions) into one of NBUF
// accumulators in tensor memory; the four epilogue warps add it, times its two
// scales, to fp32 sums in registers: lane = column of B, register = row. The
// row's scale differs per register and comes from the lane that loaded it.
//
// Roles: warp 0 TMA producer, warp 1 MMA issue, warps 2-5 epilogue. All waits
// are bounded.
#include "fp8_common.cuh"

namespace gf {
namespace {

constexpr int kThreadsNarrow = 192;
constexpr int kEpiThreads = 128;
constexpr int kBBytes = 128 * 128;

constexpr int narrow_stages(int tr, bool dual) {
  const int stage = (dual ? 2 : 1) * kBBytes + tr * 128;
  const int left = kSmemPerCta - kSmemAlignSlack - kSmemCtrlBytes - 2 * (kFp8MaxGroups + 2) * 4 - 2048;
  return left / stage > 12 ? 12 : left / stage;
}

template <int TR, bool DUAL>
struct NarrowCfg {
  static constexpr int kStageBytes = (DUAL ? 2 : 1) * kBBytes + TR * 128;
  static constexpr int kStages = narrow_stages(TR, DUAL);
  static constexpr int kTableBytes = 2 * (kFp8MaxGroups + 2) * 4;
  static constexpr int kAccCols = (DUAL ? 2 : 1) * TR;
  // accumulators in flight: up to 4, within the 512 columns of tensor memory
  static constexpr int kBufs = 512 / kAccCols > 4 ? 4 : 512 / kAccCols;
  static constexpr int kTmemCols = kBufs * kAccCols < 32     ? 32
                                   : kBufs * kAccCols <= 64  ? 64
                                   : kBufs * kAccCols <= 128 ? 128
                                   : kBufs * kAccCols <= 256 ? 256
                                                             : 512;
  static constexpr int kSmemBytes =
      kSmemAlignSlack + kStages * kStageBytes + kSmemCtrlBytes + kTableBytes + 2048;
  static_assert(16 * kStages + 16 * kBufs + 32 <= kSmemCtrlBytes, "control region");
  static_assert(kSmemBytes <= kSmemPerCta && kStages >= 3, "shared memory budget");
};

// columns [col, col + TR) of the accumulator -> 32-bit registers
template <int TR>
__device__ __forceinline__ void load_acc(uint32_t taddr, uint32_t (&r)[TR]) {
  if constexpr (TR == 16) {
    tmem_ld_32x32b_x16(taddr, r);
    tmem_ld_wait_tied(r);
  } else {
    tmem_ld_32x32b_x32(taddr, r);
    tmem_ld_wait_tied(r);
  }
}

template <typename T, int TR, bool DUAL>
__global__ void __launch_bounds__(kThreadsNarrow, 1)
    fp8_narrow_kernel(const __grid_constant__ CUtensorMap tmA,
                      const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmB2, const Fp8Params p) {
  using C = NarrowCfg<TR, DUAL>;
  constexpr int S = C::kStages;
  constexpr int CH = TR < 32 ? TR : 32;  // accumulator columns per load
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t ctrl = base + S * C::kStageBytes;
  uint8_t* gctrl = gbase + S * C::kStageBytes;
  const uint32_t full0 = ctrl, empty0 = ctrl + 8u * S;
  const uint32_t tfull0 = ctrl + 16u * S, tempty0 = tfull0 + 8u * C::kBufs;
  const uint32_t done_bar = tempty0 + 8u * C::kBufs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gctrl + 16 * S + 16 * C::kBufs + 8);
  volatile int* abort_flag =
      reinterpret_cast<volatile int*>(gctrl + 16 * S + 16 * C::kBufs + 12);
  GroupTable table;
  table.row0 = reinterpret_cast<int32_t*>(gctrl + kSmemCtrlBytes);
  table.tile0 = table.row0 + kFp8MaxGroups + 2;
  uint32_t* warp_mag = reinterpret_cast<uint32_t*>(gctrl + kSmemCtrlBytes + C::kTableBytes);

  const int warp = threadIdx.x >> 5;
  const uint32_t lane = lane_id();

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8u * s, 1);
      mbar_init(empty0 + 8u * s, 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(tfull0 + 8u * b, 1);
      mbar_init(tempty0 + 8u * b, 4);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    if (p.num_k_blocks > 0) {
      prefetch_tmap(&tmA);
      prefetch_tmap(&tmB);
      if (DUAL) prefetch_tmap(&tmB2);
    }
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  grid_dep_wait();
  grid_dep_launch();
  const int col_tiles = (p.N + 127) / 128;
  build_group_table(p, table, TR, col_tiles);
  const int num_tiles = table.tile0[p.groups + 1];
  bool aborted = false;

  // tile t: its group, first row, rows and first column of B
  auto tile_at = [&](int t, int& g, int& row, int& rows, int& nt) {
    g = group_of_tile(table, p.groups, t);
    const int first = table.row0[g], last = table.row0[g + 1];
    const int row_tiles = (last - first + TR - 1) / TR;
    const int i = t - table.tile0[g];
    nt = i / row_tiles;  // the row tiles of one B panel follow each other: it stays in L2
    row = first + (i - nt * row_tiles) * TR;
    rows = min(TR, last - row);
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int loads = 0;
      bool ok = true;
      int issued[S];
#pragma unroll
      for (int s = 0; s < S; ++s) issued[s] = -1;
      for (int t = blockIdx.x; t < num_tiles && ok; t += gridDim.x) {
        int g, row, rows, nt;
        tile_at(t, g, row, rows, nt);
        const int nkb = g < p.groups ? p.num_k_blocks : 0;
        const int brow = g * p.N + nt * 128;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait_bounded(empty0 + 8u * stage, phase ^ 1u, abort_flag, p.wait_limit_ns)) {
            fp8_raise(p, abort_flag, ST_TIMEOUT_PRODUCER);
            aborted = true;
            ok = false;
            break;
          }
          ++loads;
          if (loads != p.drop_load) {
            const uint32_t fb = full0 + 8u * stage;
            const uint32_t dst = base + stage * C::kStageBytes;
            mbar_arrive_expect_tx(fb, C::kStageBytes);
            tma_load_2d(dst, &tmB, fb, kb * 128, brow);
            if (DUAL) tma_load_2d(dst + kBBytes, &tmB2, fb, kb * 128, brow);
            tma_load_2d(dst + (DUAL ? 2 : 1) * kBBytes, &tmA, fb, kb * 128, row);
            issued[stage] = static_cast<int>(phase);
          }
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
#pragma unroll
      for (int s = 0; s < S; ++s)
        if (issued[s] >= 0 && !mbar_wait_bounded(full0 + 8u * s, static_cast<uint32_t>(issued[s]),
                                                 nullptr, p.wait_limit_ns))
          fp8_raise(p, abort_flag, ST_TIMEOUT_DRAIN);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3(128, TR);
      int stage = 0;
      uint32_t phase = 0;
      int buf = 0;
      uint32_t bphase = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < num_tiles && ok; t += gridDim.x) {
        int g, row, rows, nt;
        tile_at(t, g, row, rows, nt);
        const int nkb = g < p.groups ? p.num_k_blocks : 0;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait_bounded(tempty0 + 8u * buf, bphase ^ 1u, abort_flag, p.wait_limit_ns)) {
            fp8_raise(p, abort_flag, ST_TIMEOUT_MMA_TMEM);
            aborted = true;
            ok = false;
            break;
          }
          if (!mbar_wait_bounded(full0 + 8u * stage, phase, abort_flag, p.wait_limit_ns)) {
            fp8_raise(p, abort_flag, ST_TIMEOUT_MMA_SMEM);
            aborted = true;
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sB = base + stage * C::kStageBytes;
          const uint32_t sA = sB + (DUAL ? 2 : 1) * kBBytes;
          const uint32_t d = tmem_base + static_cast<uint32_t>(buf * C::kAccCols);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t adesc = sdesc_sw128(sA + kk * 32, 16, 1024);
            umma_f8(d, sdesc_sw128(sB + kk * 32, 16, 1024), adesc, idesc, kk != 0);
            if (DUAL)
              umma_f8(d + TR, sdesc_sw128(sB + kBBytes + kk * 32, 16, 1024), adesc, idesc,
                      kk != 0);
          }
          umma_commit(empty0 + 8u * stage);
          umma_commit(tfull0 + 8u * buf);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
          if (++buf == C::kBufs) {
            buf = 0;
            bphase ^= 1u;
          }
        }
      }
      umma_commit(done_bar);
      if (!mbar_wait_bounded(done_bar, 0, nullptr, p.wait_limit_ns))
        fp8_raise(p, abort_flag, ST_TIMEOUT_DRAIN);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;  // tensor-memory lane quarter
    const int col = 32 * q + static_cast<int>(lane);  // this thread's column of the tile
    constexpr int SL = (TR + 31) / 32;  // row scales held per lane
    int buf = 0;
    uint32_t bphase = 0;
    const int KB = p.num_k_blocks;
    for (int t = blockIdx.x; t < num_tiles; t += gridDim.x) {
      int g, row, rows, nt;
      tile_at(t, g, row, rows, nt);
      const int nkb = g < p.groups ? KB : 0;
      const float* as = p.a_scale + static_cast<int64_t>(row) * KB;
      const int64_t b_at = (static_cast<int64_t>(g) * p.num_n_blocks + nt) * KB;
      float acc[TR], acc2[DUAL ? TR : 1];
#pragma unroll
      for (int j = 0; j < TR; ++j) acc[j] = 0.0f;
      if constexpr (DUAL) {
#pragma unroll
        for (int j = 0; j < TR; ++j) acc2[j] = 0.0f;
      }
      bool ok = true;
      for (int kb = 0; kb < nkb; ++kb) {
        float sa[SL];
#pragma unroll
        for (int i = 0; i < SL; ++i) {
          const int r = 32 * i + static_cast<int>(lane);
          sa[i] = r < rows ? as[static_cast<int64_t>(r) * KB + kb] : 0.0f;
        }
        const float sb = p.b_scale[b_at + kb];
        const float sb2 = DUAL ? p.b2_scale[b_at + kb] : 0.0f;
        ok = mbar_wait_bounded(tfull0 + 8u * buf, bphase, abort_flag, p.wait_limit_ns);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(32 * q) << 16) +
                               static_cast<uint32_t>(buf * C::kAccCols);
#pragma unroll
        for (int c = 0; c < TR; c += CH) {
          uint32_t v[CH];
          load_acc<CH>(taddr + c, v);
#pragma unroll
          for (int j = 0; j < CH; ++j)
            acc[c + j] = fmaf(__uint_as_float(v[j]) * sb,
                              __shfl_sync(0xFFFFFFFFu, sa[c / 32], j), acc[c + j]);
          if constexpr (DUAL) {
            load_acc<CH>(taddr + TR + c, v);
#pragma unroll
            for (int j = 0; j < CH; ++j)
              acc2[c + j] = fmaf(__uint_as_float(v[j]) * sb2,
                                 __shfl_sync(0xFFFFFFFFu, sa[c / 32], j), acc2[c + j]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty0 + 8u * buf);
        if (++buf == C::kBufs) {
          buf = 0;
          bphase ^= 1u;
        }
      }
      // (the epilog with a barrier of all epilogue warps agrees on the outcome)
      if constexpr (DUAL) ok = !named_bar_red_or(1, kEpiThreads, !ok);
      if (!ok) {
        fp8_raise(p, abort_flag, ST_TIMEOUT_EPILOGUE);
        aborted = true;
        break;
      }
      const int n = nt * 128 + col;
      if constexpr (!DUAL) {
        T* out = static_cast<T*>(p.out) + static_cast<int64_t>(row) * p.N + n;
        if (n < p.N) {
#pragma unroll
          for (int j = 0; j < TR; ++j)
            if (j < rows) out[static_cast<int64_t>(j) * p.N] = Pair16<T>::round(acc[j]);
        }
      } else {
        // h, and its largest magnitude over the tile's 128 columns, per row
#pragma unroll
        for (int j = 0; j < TR; ++j) {
          acc[j] = n < p.N ? silu_mul(acc[j], acc2[j]) : 0.0f;
          const uint32_t mag = __reduce_max_sync(0xFFFFFFFFu, finite_mag_bits(acc[j]));
          if (lane == 0) warp_mag[q * TR + j] = mag;
        }
        named_bar_sync(1, kEpiThreads);
        uint8_t* out = static_cast<uint8_t*>(p.out) + static_cast<int64_t>(row) * p.N + n;
        float* os = p.out_scale + static_cast<int64_t>(row) * p.num_n_blocks + nt;
#pragma unroll
        for (int j = 0; j < TR; ++j) {
          const uint32_t mag = max(max(warp_mag[j], warp_mag[TR + j]),
                                   max(warp_mag[2 * TR + j], warp_mag[3 * TR + j]));
          float inv;
          const float sc = e4m3_scale(mag, inv);
          if (j < rows) {
            if (n < p.N)
              out[static_cast<int64_t>(j) * p.N] = static_cast<uint8_t>(e4m3x2(acc[j], 0.0f, inv));
            if (col == 0) os[static_cast<int64_t>(j) * p.num_n_blocks] = sc;
          }
        }
        named_bar_sync(1, kEpiThreads);  // warp_mag is read before the next tile writes it
      }
    }
  }

  // a CTA that gave up may still have loads in flight towards its shared memory
  if (__syncthreads_or(aborted ? 1 : 0) || *abort_flag) sleep_ns(200000);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

template <typename T, int TR, bool DUAL>
cudaError_t launch_instance_fp8(const Fp8LaunchArgs& a) {
  auto kernel = fp8_narrow_kernel<T, TR, DUAL>;
  constexpr int smem = NarrowCfg<TR, DUAL>::kSmemBytes;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.grid, 1, 1);
  cfg.blockDim = dim3(kThreadsNarrow, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = a.pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, *a.tmA, *a.tmB, *a.tmB2, *a.params);
}

}  // namespace

int fp8_narrow_stages(int tile_rows, int dual) { return narrow_stages(tile_rows, dual != 0); }

cudaError_t launch_fp8_narrow(const Fp8LaunchArgs& a) {
  if (a.dual) {
    switch (a.tile_rows) {
      case 16: return launch_instance_fp8<__half, 16, true>(a);
      case 64: return launch_instance_fp8<__half, 64, true>(a);
    }
    return cudaErrorInvalidValue;
  }
  switch (a.tile_rows) {
    case 16:
      return a.bf16 ? launch_instance_fp8<__nv_bfloat16, 16, false>(a)
                    : launch_instance_fp8<__half, 16, false>(a);
    case 64:
      return a.bf16 ? launch_instance_fp8<__nv_bfloat16, 64, false>(a)
                    : launch_instance_fp8<__half, 64, false>(a);
  }
  return cudaErrorInvalidValue;
}

}  // namespace gf
