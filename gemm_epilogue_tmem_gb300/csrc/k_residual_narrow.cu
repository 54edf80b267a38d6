// out = act(A B + bias) + residual for few rows (the tokens of a serving loop): a
// tile is 128 columns times TR rows, with B on the tensor core's 128-row side (D =
// B^T A^T), so that few rows cost no more tensor work than they need and a CTA streams
// one operand, B, from HBM, whose rate bounds the product (one row, 5120 columns, k =
// 17408: 29.8 us, 6.0 TB/s; by the single-CTA kernel 47).
//
// Tiles that leave SMs idle are shared by a cluster of CTAs, each with a run of their
// k-blocks: each CTA puts its fp32 partial sums into its shared memory (the idle ring),
// and each sums a part of the rows over all of them, in k order, through distributed
// shared memory, and finishes those. (Through a workspace in HBM, joined by the last
// CTA to finish: 48 rows, 5120 columns, k = 17408 39 us, so 35.) From shared memory a thread
// takes eight columns of a row, whose residual is on its way since the start.
//
// Roles: warp 0 TMA producer, warp 1 MMA issue (64-wide k-blocks, four K = 16
// instructions each), warps 2-5 epilogue. All waits are bounded.
#include "gemm_kernel.cuh"
#include "residual_narrow.h"

namespace gf {
namespace {

constexpr int kWBytes = 128 * kBK * 2;  // a k-block of 128 columns of B
constexpr int kEpiThreads = 128;

// Two CTAs an SM (113 KB each), so that the next one's is set up, and streams, while one
// finishes; their stages together cover the HBM latency.
template <int TR>
struct NarrowCfg {
  static constexpr int kStageBytes = kWBytes + TR * kBK * 2;
  static constexpr int kBudget = 113 * 1024 - kSmemAlignSlack - kSmemCtrlBytes;
  static constexpr int kStages = kBudget / kStageBytes;
  static constexpr int kSmemBytes = kSmemAlignSlack + kSmemCtrlBytes + kStages * kStageBytes;
  static constexpr int kTmemCols = TR < 32 ? 32 : TR;
  static_assert(kStages >= 4 && 16 * kStages + 64 <= kSmemCtrlBytes, "shared memory");
  static_assert(TR * 128 * 4 <= kStages * kStageBytes, "partial sums in the ring");
};

// 16 columns of 32 lanes; thread t gets lane (base lane + t)
__device__ __forceinline__ void tmem_ld_16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tie_16(uint32_t* r) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

__device__ __forceinline__ float4 ld_shared_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <typename T, int TR, bool B_MN>
__global__ void __launch_bounds__(kThreads, 2)
    residual_narrow_kernel(const __grid_constant__ CUtensorMap tmA,
                           const __grid_constant__ CUtensorMap tmB, const GemmParams p) {
  using C = NarrowCfg<TR>;
  constexpr int S = C::kStages;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t ctrl = base + S * C::kStageBytes;
  uint8_t* gctrl = smem_raw + (ctrl - raw);
  const uint32_t full0 = ctrl, empty0 = ctrl + 8u * S;
  const uint32_t done_bar = ctrl + 16u * S;    // the products are complete
  const uint32_t joined = done_bar + 8u;       // every CTA's partial sums are in place
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gctrl + 16 * S + 16);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gctrl + 16 * S + 20);

  const int warp = threadIdx.x >> 5;
  const uint32_t lane = lane_id();
  const int splits = p.k_splits;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8u * s, 1);
      mbar_init(empty0 + 8u * s, 1);
    }
    mbar_init(done_bar, 1);
    mbar_init(joined, static_cast<uint32_t>(splits));
    *abort_flag = 0;
    fence_mbar_init();
    if (p.num_k_blocks > 0) {
      prefetch_tmap(&tmA);
      prefetch_tmap(&tmB);
    }
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  if (splits > 1) cluster_sync();  // the others' barriers are there
  tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  grid_dep_wait();
  grid_dep_launch();
  bool aborted = false;

  // a CTA has one tile, a cluster's CTAs the same one; the row tiles of one panel of B
  // follow each other: it stays in L2
  const int rank = splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = static_cast<int>(blockIdx.x) / splits;
  const int nt = tile / p.num_m_blocks;
  const int row0 = (tile - nt * p.num_m_blocks) * TR, n0 = nt * 128;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.num_k_blocks) * rank / splits);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.num_k_blocks) * (rank + 1) / splits);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0, issued_phase = 0;  // bit s: a load of stage s, its phase
      const int nbox = B_MN ? min(2, (p.N - n0 + 63) / 64) : 1;
      const uint32_t bytes = TR * kBK * 2 + (B_MN && !p.b_mn_3d ? nbox * 64 * kBK * 2 : kWBytes);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait_bounded(empty0 + 8u * stage, phase ^ 1u, abort_flag, p.wait_limit_ns)) {
          raise_error(p, abort_flag, ST_TIMEOUT_PRODUCER);
          aborted = true;
          break;
        }
        if (kb - kb0 + 1 != p.drop_load) {
          const uint32_t fb = full0 + 8u * stage, w = base + stage * C::kStageBytes;
          mbar_arrive_expect_tx(fb, bytes);
          if (B_MN && p.b_mn_3d) {
            tma_load_3d(w, &tmB, fb, 0, kb * kBK, n0 / 64);
          } else if (B_MN) {
            for (int j = 0; j < nbox; ++j)
              tma_load_2d(w + j * (64 * kBK * 2), &tmB, fb, n0 + 64 * j, kb * kBK);
          } else {
            tma_load_2d(w, &tmB, fb, kb * kBK, n0);
          }
          tma_load_2d(w + kWBytes, &tmA, fb, kb * kBK, row0);
          issued |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
        }
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // every load issued must land before the CTA may exit
      for (int s = 0; s < S; ++s)
        if ((issued >> s & 1u) &&
            !mbar_wait_bounded(full0 + 8u * s, issued_phase >> s & 1u, nullptr, p.wait_limit_ns))
          raise_error(p, abort_flag, ST_TIMEOUT_DRAIN);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    if (lane == 0) {
      // (bit 15: the first operand, here B's columns, lies MN-major)
      constexpr uint32_t idesc = idesc_f16(kBf16, false, 128, TR) | (B_MN ? 1u << 15 : 0u);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait_bounded(full0 + 8u * stage, phase, abort_flag, p.wait_limit_ns)) {
          raise_error(p, abort_flag, ST_TIMEOUT_MMA_SMEM);
          aborted = true;
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t w = base + stage * C::kStageBytes;
#pragma unroll
        for (int kk = 0; kk < kBK / 16; ++kk) {
          // B's columns: K-major 32 bytes along the swizzled row; MN-major 16 rows of
          // 128 bytes, 64-column chunks 8 KB apart
          const uint64_t wdesc = B_MN ? sdesc_sw128(w + kk * 2048, 64 * kBK * 2, 1024)
                                      : sdesc_sw128(w + kk * 32, 16, 1024);
          const uint64_t adesc = sdesc_sw128(w + kWBytes + kk * 32, 16, 1024);
          umma_f16(tmem_base, wdesc, adesc, idesc, kb != kb0 || kk != 0 ? 1u : 0u);
        }
        umma_commit(empty0 + 8u * stage);
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // (all products issued must finish before tensor memory is freed; those of a
      // launch that gave up are not the sum, and nothing is taken from them)
      umma_commit(done_bar);
      if (!mbar_wait_bounded(done_bar, 0, nullptr, p.wait_limit_ns) || !ok)
        raise_error(p, abort_flag, ST_TIMEOUT_DRAIN);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;  // tensor-memory lane quarter
    const int ep = static_cast<int>(threadIdx.x) - 64;
    const int rows = min(TR, p.M - row0);
    // this CTA's rows of the tile, eight columns a thread: thread ep has columns
    // 8 (ep % 16) .. of every eighth row, from its ep / 16th on
    const int share = (rows + splits - 1) / splits;
    const int j_end = min(rows, (rank + 1) * share);
    const int j_mine = rank * share + ep / 16, n = n0 + 8 * (ep % 16);
    constexpr int kItems = TR / 8;
    const bool in = n < p.N;
    auto at = [&](int i) { return static_cast<int64_t>(row0 + j_mine + 8 * i) * p.N + n; };
    uint4 res[kItems], bias8 = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < kItems; ++i)
      if (in && j_mine + 8 * i < j_end)
        res[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.residual) + at(i));
    if (p.bias != nullptr && in)
      bias8 = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.bias) + n);
    bool ok = mbar_wait_bounded(done_bar, 0, abort_flag, p.wait_limit_ns);
    // all epilogue warps agree on the outcome (barriers follow)
    ok = !named_bar_red_or(1, kEpiThreads, !ok);
    if (!ok) {
      raise_error(p, abort_flag, ST_TIMEOUT_EPILOGUE);
      aborted = true;
    } else {
      // partial sums into the ring, which has been read: [row][128 columns]
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
      const uint32_t mine = base + 4u * (32u * static_cast<uint32_t>(q) + lane);
#pragma unroll
      for (int j0 = 0; j0 < TR; j0 += 16) {
        uint32_t v[16];
        if (p.num_k_blocks > 0) {
          tmem_ld_16(taddr + j0, v);
          tmem_ld_wait();
          tie_16(v);
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = 0u;  // nothing to multiply
        }
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (j0 + j < rows) st_shared_u32(mine + 512u * static_cast<uint32_t>(j0 + j), v[j]);
      }
      tc_fence_before();
      named_bar_sync(1, kEpiThreads);
      if (splits > 1) {
        if (ep < splits) mbar_arrive_remote(mapa_shared(joined, static_cast<uint32_t>(ep)));
        if (!mbar_wait_bounded_cluster(joined, 0, abort_flag, p.wait_limit_ns)) {
          raise_error(p, abort_flag, ST_TIMEOUT_EPILOGUE);
          aborted = true;
        }
      }
      float b8[8];
      unpack8<T>(bias8, b8);
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        if (in && !aborted && j_mine + 8 * i < j_end) {
          const uint32_t from = base + 512u * static_cast<uint32_t>(j_mine + 8 * i) +
                                32u * static_cast<uint32_t>(ep % 16);
          float4 lo[kNarrowMaxSplits], hi[kNarrowMaxSplits];
#pragma unroll
          for (int c = 0; c < kNarrowMaxSplits; ++c) {
            if (c < splits) {
              const uint32_t there = splits > 1 ? mapa_shared(from, static_cast<uint32_t>(c)) : from;
              lo[c] = ld_shared_cluster(there);
              hi[c] = ld_shared_cluster(there + 16u);
            }
          }
          float z[8] = {lo[0].x, lo[0].y, lo[0].z, lo[0].w, hi[0].x, hi[0].y, hi[0].z, hi[0].w};
#pragma unroll
          for (int c = 1; c < kNarrowMaxSplits; ++c) {
            if (c < splits) {
              const float x[8] = {lo[c].x, lo[c].y, lo[c].z, lo[c].w, hi[c].x, hi[c].y, hi[c].z, hi[c].w};
#pragma unroll
              for (int j = 0; j < 8; ++j) z[j] += x[j];
            }
          }
          float r8[8];
          unpack8<T>(res[i], r8);
          if (p.bias != nullptr) {
#pragma unroll
            for (int j = 0; j < 8; ++j) z[j] += b8[j];
          }
          if (p.aux_out != nullptr)
            *reinterpret_cast<uint4*>(reinterpret_cast<T*>(p.aux_out) + at(i)) =
                make_uint4(pack2<T>(z[0], z[1]), pack2<T>(z[2], z[3]), pack2<T>(z[4], z[5]),
                           pack2<T>(z[6], z[7]));
          apply_act(p.act, z);
#pragma unroll
          for (int j = 0; j < 8; ++j) z[j] += r8[j];
          *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + at(i)) =
              make_uint4(pack2<T>(z[0], z[1]), pack2<T>(z[2], z[3]), pack2<T>(z[4], z[5]),
                         pack2<T>(z[6], z[7]));
        }
      }
    }
  }

  // a CTA that gave up may still have loads in flight towards its shared memory
  if (__syncthreads_or(aborted ? 1 : 0) || *abort_flag) sleep_ns(200000);
  tc_fence_before();
  __syncthreads();
  if (splits > 1) cluster_sync();  // no CTA leaves while another reads its partial sums
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

cudaLaunchConfig_t config(int smem, int grid, int splits, int pdl, cudaStream_t stream,
                          cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = splits > 1 ? 2 : 1;
  return cfg;
}

template <int TR>
int clusters_of(int splits) {
  auto kernel = residual_narrow_kernel<__half, TR, false>;
  constexpr int smem = NarrowCfg<TR>::kSmemBytes;
  int n = 0;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = config(smem, splits, splits, 0, nullptr, attr);
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

template <typename T, int TR, bool B_MN>
cudaError_t launch_instance_of(const LaunchArgs& a) {
  auto kernel = residual_narrow_kernel<T, TR, B_MN>;
  constexpr int smem = NarrowCfg<TR>::kSmemBytes;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = config(smem, a.grid, a.params->k_splits, a.pdl, a.stream, attr);
  return cudaLaunchKernelEx(&cfg, kernel, *a.tmA, *a.tmB, *a.params);
}

template <typename T, bool B_MN>
cudaError_t launch_rows(const LaunchArgs& a) {
  switch (a.tile_n) {
    case 16: return launch_instance_of<T, 16, B_MN>(a);
    case 32: return launch_instance_of<T, 32, B_MN>(a);
    case 64: return launch_instance_of<T, 64, B_MN>(a);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

int narrow_stages(int rows) {
  return rows == 16   ? NarrowCfg<16>::kStages
         : rows == 32 ? NarrowCfg<32>::kStages
                      : NarrowCfg<64>::kStages;
}

int narrow_clusters(int rows, int splits) {
  // The query counts one CTA an SM for a kernel with tensor memory. Two are resident, so
  // that a cluster fits on half as many SMs as it has CTAs, and every SM holds two.
  auto query = [&](int n) {
    return rows == 16 ? clusters_of<16>(n) : rows == 32 ? clusters_of<32>(n) : clusters_of<64>(n);
  };
  const int twice = 2 * query(splits), packed = splits > 2 ? query((splits + 1) / 2) : twice;
  return twice > packed ? twice : packed;
}

cudaError_t launch_residual_narrow(const LaunchArgs& a) {
  if (a.bf16) return a.b_mn ? launch_rows<__nv_bfloat16, true>(a) : launch_rows<__nv_bfloat16, false>(a);
  return a.b_mn ? launch_rows<__half, true>(a) : launch_rows<__half, false>(a);
}

}  // namespace gf
