// Block-scaled e4m3 product for few rows a group: a tile is 128 columns of B
// times TR rows, with B on the tensor core's 128-row side (D = B . A^T), so
// that a tile of 16 rows costs no more tensor work than 16 rows need and the
// whole CTA streams one operand, B, from HBM.
//
// The scales vary along k, so the tensor core sums one block of 128 at a time
// (one 128-byte-swizzled stage, four K = 32 instructions) into one of kBufs
// accumulators in tensor memory; the four epilogue warps add it, times its two
// scales, to fp32 sums in registers: lane = column of B, register = row. The
// rows' scales differ per register: a warp of its own copies them into a ring
// in shared memory, from where every thread reads four at a time (taken from
// another lane by shuffles instead, the shuffles set the pace: 219 against
// 165 us on 1.07 GB of weights with 64-row tiles).
//
// CTA c has the tiles c, c + G, ... whole where those fill most of the grid's
// rounds: an SM alone takes more than its share of the HBM rate, so that the
// others make up for an idle one (one row, 12000 columns, k = 16384, 94 tiles on
// 152 SMs: 38.9 us whole, 40.1 split; 48 rows, 9000 columns, 213 tiles 57 and 72;
// 96 rows, 4096 columns, 192 tiles 56 and 47). So it has them where splitting them
// evenly would spare each CTA fewer k-blocks than the join of the parts costs (one
// row, 4096 columns, 32 tiles: k = 2048 6.9 us whole, 7.1 split; k = 2944 8.7 and
// 7.4; 5120 columns, k = 17408: 35 and 17). Otherwise they are split in units of
// one k-block: CTA c has the units [c W / G, (c + 1) W / G) of the tiles laid
// end to end. A tile that falls to several CTAs is summed by the last
// of them to finish, over the partial sums in the plan's workspace in k order:
// no CTA waits for another, and the sum's order does not depend on which is last.
//
// Roles: warp 0 TMA producer, warp 1 MMA issue, warps 2-5 epilogue, warp 6
// scale loads. All waits are bounded.
#include "fp8_common.cuh"

namespace gf {
namespace {

constexpr int kThreadsNarrow = 224;
constexpr int kEpiThreads = 128;
constexpr int kBBytes = 128 * 128;
constexpr int kScaleGroup = 8;  // blocks whose scales come together
constexpr int kRing = 2;        // such groups in flight

// shared memory besides the stages and the table of groups
constexpr int narrow_fixed(int tr) {
  return kSmemAlignSlack + kSmemCtrlBytes + 4 * tr * 4 + kRing * kScaleGroup * (tr + 4) * 4;
}
constexpr int narrow_table(int groups) { return 2 * (groups + 2) * 4; }
// 16-row tiles: two CTAs fit on an SM (113 KB each, with the table of 128
// groups), so that the next launch's are set up and waiting when this one ends;
// their 90 KB of stages still cover the HBM latency (45 KB at the copy rate).
// 64-row tiles take the whole SM.
constexpr int kSmemHalf = 113 * 1024;
constexpr int narrow_stages(int tr, bool dual) {
  const int stage = (dual ? 2 : 1) * kBBytes + tr * 128;
  const int left = tr == 16 ? kSmemHalf - narrow_fixed(tr) - narrow_table(128)
                            : kSmemPerCta - narrow_fixed(tr) - narrow_table(kFp8MaxGroups);
  return left / stage > 12 ? 12 : left / stage;
}

template <int TR, bool DUAL>
struct NarrowCfg {
  static constexpr int kStageBytes = (DUAL ? 2 : 1) * kBBytes + TR * 128;
  static constexpr int kStages = narrow_stages(TR, DUAL);
  static constexpr int kSlot = TR + 4;  // floats of a ring slot: rows, one or two columns' scales
  static constexpr int kAccCols = (DUAL ? 2 : 1) * TR;
  // accumulators in flight: up to 4, within the 512 columns of tensor memory
  static constexpr int kBufs = 512 / kAccCols > 4 ? 4 : 512 / kAccCols;
  static constexpr int kTmemCols = kBufs * kAccCols <= 64    ? 64
                                   : kBufs * kAccCols <= 128 ? 128
                                   : kBufs * kAccCols <= 256 ? 256
                                                             : 512;
  static constexpr int kSmemBytes = narrow_fixed(TR) + kStages * kStageBytes;  // + the table
  static_assert(16 * kStages + 16 * kBufs + 16 + 16 * kRing <= kSmemCtrlBytes, "control region");
  static_assert(kSmemBytes + narrow_table(kFp8MaxGroups) <= kSmemPerCta && kStages >= 3,
                "shared memory budget");
};

// A run of k-blocks of one tile.
struct Piece {
  int tile, kb0, kb1;
};

// The pieces of a CTA, in order: `step` == 0: `at` .. `end` are units (k-blocks
// of the tiles laid end to end); else whole tiles `at`, `at` + step, ...
struct Pieces {
  int64_t at, end;
  int KB, step;
  __device__ __forceinline__ bool next(Piece& p) {
    if (at >= end) return false;
    if (step != 0) {
      p = {static_cast<int>(at), 0, KB};
      at += step;
      return true;
    }
    p.tile = static_cast<int>(at / KB);
    p.kb0 = static_cast<int>(at - static_cast<int64_t>(p.tile) * KB);
    const int64_t left = end - at;
    p.kb1 = left < KB - p.kb0 ? p.kb0 + static_cast<int>(left) : KB;
    at += p.kb1 - p.kb0;
    return true;
  }
};

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

__device__ __forceinline__ void tmem_ld_wait_tied_x16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

template <int CH>
__device__ __forceinline__ void load_acc(uint32_t taddr, uint32_t (&r)[CH]) {
  if constexpr (CH == 16) {
    tmem_ld_32x32b_x16(taddr, r);
    tmem_ld_wait_tied_x16(r);
  } else {
    tmem_ld_32x32b_x32(taddr, r);
    tmem_ld_wait_tied(r);
  }
}

// v * s, two columns at a time
__device__ __forceinline__ uint64_t mul2(uint32_t v0, uint32_t v1, uint64_t s) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(v0), "r"(v1));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(s));
  return v;
}
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t v, uint64_t s) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(s));
}

// acc += (an accumulator's CH columns) * sb * (their rows' scales at `sa`)
template <int CH>
__device__ __forceinline__ void add_scaled(uint64_t* acc, const uint32_t (&v)[CH], uint64_t sb,
                                           const float* sa) {
#pragma unroll
  for (int j = 0; j < CH; j += 4) {
    const float4 s = *reinterpret_cast<const float4*>(sa + j);
    fma2(acc[j / 2], mul2(v[j], v[j + 1], sb), pack2(s.x, s.y));
    fma2(acc[j / 2 + 1], mul2(v[j + 2], v[j + 3], sb), pack2(s.z, s.w));
  }
}

template <typename T, int TR, bool DUAL>
__global__ void __launch_bounds__(kThreadsNarrow, TR == 16 ? 2 : 1)
    fp8_narrow_kernel(const __grid_constant__ CUtensorMap tmA,
                      const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmB2, const Fp8Params p) {
  using C = NarrowCfg<TR, DUAL>;
  constexpr int S = C::kStages;
  constexpr int CH = TR < 32 ? TR : 32;  // accumulator columns per load
  constexpr int NACC = (DUAL ? 2 : 1) * TR / 2;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t ctrl = base + S * C::kStageBytes;
  uint8_t* gctrl = smem_raw + (ctrl - raw);
  const uint32_t full0 = ctrl, empty0 = ctrl + 8u * S;
  const uint32_t tfull0 = ctrl + 16u * S, tempty0 = tfull0 + 8u * C::kBufs;
  const uint32_t sfull0 = tempty0 + 8u * C::kBufs, sempty0 = sfull0 + 8u * kRing;
  const uint32_t done_bar = sempty0 + 8u * kRing;
  volatile uint32_t* words =
      reinterpret_cast<volatile uint32_t*>(gctrl + (done_bar - ctrl) + 8);
  uint32_t* tmem_slot = const_cast<uint32_t*>(words);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(words + 1);
  // the ring first: its slots are read 16 bytes at a time
  float* ring = reinterpret_cast<float*>(gctrl + kSmemCtrlBytes);
  uint32_t* warp_mag = reinterpret_cast<uint32_t*>(ring + kRing * kScaleGroup * C::kSlot);
  GroupTable table;
  table.row0 = reinterpret_cast<int32_t*>(warp_mag + 4 * TR);
  table.tile0 = table.row0 + p.groups + 2;
  __shared__ int last_flag;

  const int warp = threadIdx.x >> 5;
  const uint32_t lane = lane_id();
  const int KB = p.num_k_blocks;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8u * s, 1);
      mbar_init(empty0 + 8u * s, 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(tfull0 + 8u * b, 1);
      mbar_init(tempty0 + 8u * b, 4);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(sfull0 + 8u * i, 32);
      mbar_init(sempty0 + 8u * i, 4);
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
  const int product_tiles = KB > 0 ? table.tile0[p.groups] : 0;  // the others are zeros
  bool aborted = false;

  const int cta = static_cast<int>(blockIdx.x), grid = static_cast<int>(gridDim.x);
  const int ctas = fp8_split_ctas(product_tiles, KB, grid, TR, DUAL);
  const bool whole = ctas == 0;
  const int64_t units = static_cast<int64_t>(product_tiles) * KB;
  auto first_unit = [&](int c) { return units * c / ctas; };
  Pieces mine;
  mine.KB = KB;
  mine.step = whole ? grid : 0;
  mine.at = whole ? cta : cta < ctas ? first_unit(cta) : 0;
  mine.end = whole ? product_tiles : cta < ctas ? first_unit(cta + 1) : 0;

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

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const uint32_t e = elect_one();
    int stage = 0;
    uint32_t phase = 0;
    int loads = 0;
    bool ok = true;
    uint32_t issued = 0, issued_phase = 0;  // bit s: a load of stage s, and its phase
    Piece u;
    while (ok && mine.next(u)) {
      int g, row, rows, nt;
      tile_at(u.tile, g, row, rows, nt);
      const int b_row = g * p.N + nt * 128;
      for (int kb = u.kb0; kb < u.kb1; ++kb) {
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
          const uint32_t dst = base + stage * C::kStageBytes;
          if (e) mbar_arrive_expect_tx(fb, C::kStageBytes);
          __syncwarp();
          tma_load_f8<false>(dst, &tmB, fb, kb * 128, b_row, e);
          if (DUAL) tma_load_f8<false>(dst + kBBytes, &tmB2, fb, kb * 128, b_row, e);
          tma_load_f8<false>(dst + (DUAL ? 2 : 1) * kBBytes, &tmA, fb, kb * 128, row, e);
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
      if ((issued >> s & 1u) && !mbar_wait_bounded(full0 + 8u * s, issued_phase >> s & 1u, nullptr,
                                                   p.wait_limit_ns))
        fp8_raise(p, abort_flag, ST_TIMEOUT_DRAIN);
    __syncwarp();
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    constexpr uint32_t idesc = idesc_e4m3(128, TR);
    const uint32_t e = elect_one();
    const uint64_t desc0 = sdesc_sw128(base, 16, 1024);
    int stage = 0, buf = 0;
    uint32_t phase = 0, bphase = 0;
    bool ok = true;
    const int64_t blocks =
        whole ? (mine.end - mine.at + grid - 1) / grid * KB : mine.end - mine.at;
    for (int64_t i = blocks; i > 0; --i) {
      ok = mbar_wait_bounded(tempty0 + 8u * buf, bphase ^ 1u, abort_flag, p.wait_limit_ns);
      if (!__all_sync(0xFFFFFFFFu, ok)) {
        fp8_raise(p, abort_flag, ST_TIMEOUT_MMA_TMEM);
        aborted = true;
        break;
      }
      ok = mbar_wait_bounded(full0 + 8u * stage, phase, abort_flag, p.wait_limit_ns);
      if (!__all_sync(0xFFFFFFFFu, ok)) {
        fp8_raise(p, abort_flag, ST_TIMEOUT_MMA_SMEM);
        aborted = true;
        break;
      }
      tc_fence_after();
      // (a descriptor's address field counts 16 bytes)
      const uint64_t bdesc = desc0 + static_cast<uint64_t>(stage * (C::kStageBytes / 16));
      const uint64_t adesc = bdesc + (DUAL ? 2 : 1) * kBBytes / 16;
      const uint32_t d = tmem_base + static_cast<uint32_t>(buf * C::kAccCols);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        umma_f8<false>(d, bdesc + 2 * kk, adesc + 2 * kk, idesc, kk != 0, e);
        if (DUAL)
          umma_f8<false>(d + TR, bdesc + kBBytes / 16 + 2 * kk, adesc + 2 * kk, idesc, kk != 0, e);
      }
      umma_commit_f8<false>(tfull0 + 8u * buf, e);
      umma_commit_f8<false>(empty0 + 8u * stage, e);
      if (++stage == S) {
        stage = 0;
        phase ^= 1u;
      }
      if (++buf == C::kBufs) {
        buf = 0;
        bphase ^= 1u;
      }
    }
    umma_commit_f8<false>(done_bar, e);
    if (!mbar_wait_bounded(done_bar, 0, nullptr, p.wait_limit_ns))
      fp8_raise(p, abort_flag, ST_TIMEOUT_DRAIN);
    __syncwarp();
  } else if (warp == 6) {
    // --------------------------------------------------------- scale loads
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    const uint32_t ring_s = smem_u32(ring);
    Piece u;
    while (ok && mine.next(u)) {
      int g, row, rows, nt;
      tile_at(u.tile, g, row, rows, nt);
      const float* as = p.a_scale + static_cast<int64_t>(row + static_cast<int>(lane)) * KB;
      // lanes 0 and 1: the scales of the tile's columns of B and of B2
      const float* bs = (DUAL && lane == 1 ? p.b2_scale : p.b_scale) +
                        (static_cast<int64_t>(g) * p.num_n_blocks + nt) * KB;
      for (int kb0 = u.kb0; kb0 < u.kb1; kb0 += kScaleGroup) {
        ok = mbar_wait_bounded(sempty0 + 8u * slot, phase ^ 1u, abort_flag, p.wait_limit_ns);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) {
          fp8_raise(p, abort_flag, ST_TIMEOUT_PRODUCER);
          aborted = true;
          break;
        }
        const int last = min(kb0 + kScaleGroup, u.kb1);
        uint32_t dst = ring_s + 4u * (C::kSlot * kScaleGroup * slot + lane);
        for (int kb = kb0; kb < last; ++kb, dst += 4u * C::kSlot) {
#pragma unroll
          for (int i = 0; i < (TR + 31) / 32; ++i) {
            const int r = 32 * i + static_cast<int>(lane);
            const bool in = r < rows;  // rows past the tile's: zero
            if (r < TR)
              cp_async_4(dst + 128u * i,
                         in ? as + static_cast<int64_t>(32 * i) * KB + kb : p.a_scale, in);
          }
          if (lane < (DUAL ? 2 : 1)) cp_async_4(dst + 4u * TR, bs + kb, true);
        }
        cp_async_arrive(sfull0 + 8u * slot);
        if (++slot == kRing) {
          slot = 0;
          phase ^= 1u;
        }
      }
    }
    cp_async_wait_all();  // no copy lands after the CTA is gone
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;  // tensor-memory lane quarter
    const int col = 32 * q + static_cast<int>(lane);  // this thread's column of the tile
    int buf = 0, slot = 0;
    uint32_t bphase = 0, sphase = 0;

    uint64_t acc[NACC];
    auto store_tile = [&](int row, int rows, int nt) {
      const int n = nt * 128 + col;
      if constexpr (!DUAL) {
        T* out = static_cast<T*>(p.out) + static_cast<int64_t>(row) * p.N + n;
        if (n < p.N) {
#pragma unroll
          for (int j = 0; j < TR; j += 2) {
            const float2 f = split2(acc[j / 2]);
            if (j < rows) out[static_cast<int64_t>(j) * p.N] = Pair16<T>::round(f.x);
            if (j + 1 < rows) out[static_cast<int64_t>(j + 1) * p.N] = Pair16<T>::round(f.y);
          }
        }
      } else {
        // h, and its largest magnitude over the tile's 128 columns, per row
#pragma unroll
        for (int j = 0; j < TR; j += 2) {
          const float2 g = split2(acc[j / 2]), v = split2(acc[(TR + j) / 2]);
          const float h0 = n < p.N ? silu_mul(g.x, v.x) : 0.0f;
          const float h1 = n < p.N ? silu_mul(g.y, v.y) : 0.0f;
          acc[j / 2] = pack2(h0, h1);
          const uint32_t m0 = __reduce_max_sync(0xFFFFFFFFu, finite_mag_bits(h0));
          const uint32_t m1 = __reduce_max_sync(0xFFFFFFFFu, finite_mag_bits(h1));
          if (lane == 0) {
            warp_mag[q * TR + j] = m0;
            warp_mag[q * TR + j + 1] = m1;
          }
        }
        named_bar_sync(1, kEpiThreads);
        uint8_t* out = static_cast<uint8_t*>(p.out) + static_cast<int64_t>(row) * p.N + n;
        float* os = p.out_scale + static_cast<int64_t>(row) * p.num_n_blocks + nt;
#pragma unroll
        for (int j = 0; j < TR; ++j) {
          const uint32_t mag = max(max(warp_mag[j], warp_mag[TR + j]),
                                   max(warp_mag[2 * TR + j], warp_mag[3 * TR + j]));
          const float2 h = split2(acc[j / 2]);
          float inv;
          const float sc = e4m3_scale(mag, inv);
          if (j < rows) {
            if (n < p.N)
              out[static_cast<int64_t>(j) * p.N] =
                  static_cast<uint8_t>(e4m3x2(j % 2 ? h.y : h.x, 0.0f, inv));
            if (col == 0) os[static_cast<int64_t>(j) * p.num_n_blocks] = sc;
          }
        }
        named_bar_sync(1, kEpiThreads);  // warp_mag is read before the next tile writes it
      }
    };

    Piece u;
    bool ok = true;
    while (mine.next(u)) {
      int g, row, rows, nt;
      tile_at(u.tile, g, row, rows, nt);
#pragma unroll
      for (int j = 0; j < NACC; ++j) acc[j] = 0ull;
      for (int left = u.kb1 - u.kb0; left > 0 && ok; left -= kScaleGroup) {
        ok = mbar_wait_bounded(sfull0 + 8u * slot, sphase, abort_flag, p.wait_limit_ns);
        const float* sc = ring + C::kSlot * kScaleGroup * slot;
        for (int kb = min(left, kScaleGroup); kb > 0; --kb, sc += C::kSlot) {
          ok = mbar_wait_bounded(tfull0 + 8u * buf, bphase, abort_flag, p.wait_limit_ns) && ok;
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint64_t sb = both(sc[TR]);
          const uint64_t sb2 = DUAL ? both(sc[TR + 1]) : sb;
          const uint32_t taddr = tmem_base + (static_cast<uint32_t>(32 * q) << 16) +
                                 static_cast<uint32_t>(buf * C::kAccCols);
#pragma unroll
          for (int c = 0; c < TR; c += CH) {
            uint32_t v[CH];
            load_acc<CH>(taddr + c, v);
            add_scaled<CH>(acc + c / 2, v, sb, sc + c);
            if constexpr (DUAL) {
              load_acc<CH>(taddr + TR + c, v);
              add_scaled<CH>(acc + (TR + c) / 2, v, sb2, sc + c);
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
      if (u.kb0 != 0 || u.kb1 != KB) {
        // a piece: its partial sums to the workspace (slot 1 of this CTA when
        // it starts the tile, else slot 0). The tile's pieces belong to
        // consecutive CTAs, from the one with the tile's first unit; the last
        // to count adds them in order
        const int64_t first = static_cast<int64_t>(u.tile) * KB;
        const int c0 = fp8_unit_owner(first, units, ctas);
        const int c1 = fp8_unit_owner(first + KB - 1, units, ctas);
        float2* ws = reinterpret_cast<float2*>(p.partials);
        float2* dst = ws + (static_cast<int64_t>(2 * cta + (u.kb0 == 0 ? 1 : 0)) * NACC) * 128 + col;
#pragma unroll
        for (int j = 0; j < NACC; ++j) __stcg(dst + j * 128, split2(acc[j]));
        __threadfence();
        named_bar_sync(1, kEpiThreads);
        if (col == 0) {
          const int done = atomicAdd(p.counters + c0, 1);
          last_flag = done == c1 - c0;
          if (done == c1 - c0) p.counters[c0] = 0;  // for the next launch
        }
        named_bar_sync(1, kEpiThreads);
        if (!last_flag) continue;
        __threadfence();
#pragma unroll
        for (int j = 0; j < NACC; ++j) acc[j] = 0ull;
        for (int c = c0; c <= c1; ++c) {
          const float2* src = ws + (static_cast<int64_t>(2 * c + (c == c0 ? 1 : 0)) * NACC) * 128 + col;
#pragma unroll
          for (int j = 0; j < NACC; ++j) {
            const float2 v = __ldcg(src + j * 128), a = split2(acc[j]);
            acc[j] = pack2(a.x + v.x, a.y + v.y);
          }
        }
      }
      store_tile(row, rows, nt);
    }
    // the rows of no group (and every row of a product over nothing)
    if (ok) {
#pragma unroll
      for (int j = 0; j < NACC; ++j) acc[j] = 0ull;
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
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

template <typename T, int TR, bool DUAL>
cudaError_t launch_narrow(const Fp8LaunchArgs& a) {
  auto kernel = fp8_narrow_kernel<T, TR, DUAL>;
  const int smem = NarrowCfg<TR, DUAL>::kSmemBytes + narrow_table(a.params->groups);
  const cudaError_t e = cudaFuncSetAttribute(
      kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
      NarrowCfg<TR, DUAL>::kSmemBytes + narrow_table(kFp8MaxGroups));
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

template <typename T, bool DUAL>
cudaError_t launch_rows(const Fp8LaunchArgs& a) {
  switch (a.tile_rows) {
    case 16: return launch_narrow<T, 16, DUAL>(a);
    case 64: return launch_narrow<T, 64, DUAL>(a);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

int fp8_narrow_stages(int tile_rows, int dual) { return narrow_stages(tile_rows, dual != 0); }

size_t fp8_narrow_partial_bytes(int tile_rows, int dual, int grid) {
  return static_cast<size_t>(grid) * 2 * (dual ? 2 : 1) * tile_rows * 128 * 4;
}

cudaError_t launch_fp8_narrow(const Fp8LaunchArgs& a) {
  if (a.dual) return launch_rows<__half, true>(a);
  return a.bf16 ? launch_rows<__nv_bfloat16, false>(a) : launch_rows<__half, false>(a);
}

}  // namespace gf
