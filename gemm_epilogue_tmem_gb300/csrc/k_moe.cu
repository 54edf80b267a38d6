// Expert routing: the stable sort of the (token, slot) pairs by expert, the
// copies of the tokens' rows to their places and back, and their gradients.
//
// Everything here is bound by HBM: the arithmetic is a few operations per
// element. Each kernel is token-driven, so that the one row that all of a
// token's slots share (x, out, d_out) passes through the chip once and only
// the topk rows per token that differ are read or written.
//
// Rows whose length is not a multiple of 16 bytes (ANY below) start at every
// even byte. Their accesses are 16 bytes all the same: stores go by the
// aligned words of the row that is written (its first and last word element by
// element), and what they need of another row is shifted out of the two
// aligned words that hold it (5003 tokens, 6 slots, 2047 columns of fp16: the
// gradient of dispatch took 87 us with 2-byte accesses).
//
// The kernels begin while the one before them, which may write what they read,
// still runs. So no load goes through the read-only path (__ldg, or const and
// __restrict__ pointers), which is for data that nobody writes while a kernel lives.
#include <type_traits>

#include "fp8.cuh"
#include "moe.h"
#include "ptx.cuh"

namespace gf {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kRankWarps = 8;        // warps that rank the slots of a chunk
constexpr uint32_t kSortCluster = 8;

template <typename K, typename... A>
cudaError_t launch_clusters(K kernel, dim3 grid, unsigned cluster, int threads, size_t smem,
                            cudaStream_t stream, int pdl, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename K, typename... A>
cudaError_t launch(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, int pdl,
                   A... args) {
  return launch_clusters(kernel, grid, 1, threads, smem, stream, pdl, args...);
}

// ------------------------------------------------------------------- the sort
// A counting sort over chunks of consecutive tokens, one CTA each: the place
// of a slot is its expert's first row, plus the kept slots of that expert in
// earlier chunks, in earlier warps of its chunk and earlier in its warp. Every
// term is a count, so the order is stable and the same in every run.
//
// The counts over all slots are made by every CTA alone, or with many slots by
// every cluster of kSortCluster CTAs for itself, a part by each, and shared
// through its distributed shared memory: one launch and no workspace (65536
// slots: 9.5 us, 11 with a kernel that counts the chunks first).

__device__ __forceinline__ int ld_cluster(uint32_t cluster_addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// --------------------------------------------------------- rows of any length
// A coherent load that the compiler may move over stores, which go to other arrays
// (a plain one stays behind them: gradient of combine, 5003 tokens, 6 slots, 2047
// columns, 57 us, with this one 54.5). Not over grid_dep_wait as long as the address
// depends on an index that was loaded after it, as the row of a slot does.
__device__ __forceinline__ uint4 load_early(const uint4* p) {
  uint4 v;
  asm("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
      : "l"(p));
  return v;
}

// The aligned 16-byte word at byte `at` of an array of `total` bytes; bytes
// outside it are zero and are not read.
__device__ __forceinline__ uint4 word_at(const uint8_t* array, int64_t at, int64_t total) {
  if (at >= 0 && at + 16 <= total) return *reinterpret_cast<const uint4*>(array + at);
  uint32_t w[4] = {0, 0, 0, 0};
  if (at >= 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (at + 2 * i < total)
        w[i / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(array + at + 2 * i))
                    << (16 * (i & 1));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The 16 bytes that begin `shift` (even, below 16) bytes into a and end in b.
// The shift is the same for all words of a row, and so for the warp: a branch
// per 4 bytes of it instead of selecting every word.
__device__ __forceinline__ uint4 shift_out(const uint4& a, const uint4& b, uint32_t shift) {
  const uint32_t r = 8u * (shift & 2u);
  switch (shift >> 2) {
    case 0:
      return make_uint4(__funnelshift_r(a.x, a.y, r), __funnelshift_r(a.y, a.z, r),
                        __funnelshift_r(a.z, a.w, r), __funnelshift_r(a.w, b.x, r));
    case 1:
      return make_uint4(__funnelshift_r(a.y, a.z, r), __funnelshift_r(a.z, a.w, r),
                        __funnelshift_r(a.w, b.x, r), __funnelshift_r(b.x, b.y, r));
    case 2:
      return make_uint4(__funnelshift_r(a.z, a.w, r), __funnelshift_r(a.w, b.x, r),
                        __funnelshift_r(b.x, b.y, r), __funnelshift_r(b.y, b.z, r));
    default:
      return make_uint4(__funnelshift_r(a.w, b.x, r), __funnelshift_r(b.x, b.y, r),
                        __funnelshift_r(b.y, b.z, r), __funnelshift_r(b.z, b.w, r));
  }
}

// The same, of this lane's word and the next lane's: a shuffle for each 4 bytes
// that the next one gives, one to four. Called by whole warps with one shift.
__device__ __forceinline__ uint4 shift_in(const uint4& a, uint32_t shift) {
  const uint32_t r = 8u * (shift & 2u);
  auto next = [](uint32_t w) { return __shfl_down_sync(0xFFFFFFFFu, w, 1); };
  switch (shift >> 2) {
    case 0: {
      const uint32_t x = next(a.x);
      return make_uint4(__funnelshift_r(a.x, a.y, r), __funnelshift_r(a.y, a.z, r),
                        __funnelshift_r(a.z, a.w, r), __funnelshift_r(a.w, x, r));
    }
    case 1: {
      const uint32_t x = next(a.x), y = next(a.y);
      return make_uint4(__funnelshift_r(a.y, a.z, r), __funnelshift_r(a.z, a.w, r),
                        __funnelshift_r(a.w, x, r), __funnelshift_r(x, y, r));
    }
    case 2: {
      const uint32_t x = next(a.x), y = next(a.y), z = next(a.z);
      return make_uint4(__funnelshift_r(a.z, a.w, r), __funnelshift_r(a.w, x, r),
                        __funnelshift_r(x, y, r), __funnelshift_r(y, z, r));
    }
    default: {
      const uint32_t x = next(a.x), y = next(a.y), z = next(a.z), v = next(a.w);
      return make_uint4(__funnelshift_r(a.w, x, r), __funnelshift_r(x, y, r),
                        __funnelshift_r(y, z, r), __funnelshift_r(z, v, r));
    }
  }
}

// acc += w f, both columns in one instruction
__device__ __forceinline__ void add_scaled(float2& acc, const float2& f, float w) {
  asm("{\n\t.reg .b64 a, b, c;\n\t"
      "mov.b64 a, {%0, %1};\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "mov.b64 c, {%4, %4};\n\t"
      "fma.rn.f32x2 a, b, c, a;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "+f"(acc.x), "+f"(acc.y)
      : "f"(f.x), "f"(f.y), "f"(w));
}

// The 16 bytes from byte `at` (even) on, out of the two aligned words around
// them; bytes outside the array are zero and are not read.
__device__ __forceinline__ uint4 bytes_at(const uint8_t* array, int64_t at, int64_t total) {
  const uint32_t shift = static_cast<uint32_t>(at) & 15u;
  return shift_out(word_at(array, at - shift, total), word_at(array, at - shift + 16, total),
                   shift);
}

// Whether every aligned word that holds an element of the row, and the word
// before and after it, lies in an array of `rows` rows of H elements: their
// loads then need no checks. So it does for all rows but the first and last.
__device__ __forceinline__ bool row_inside(int row, int rows, int H) {
  return H >= 32 && row > 0 && row < rows - 1;
}

// How a row of H 16-bit elements is cut into words of 8. Aligned: column 8 v.
// ANY: by the aligned words of the array, the first and last of which may
// hold neighbours' elements too.
template <bool ANY>
struct RowWords {
  int H;
  int lead;       // elements before the row in its first word
  int64_t start;  // first element of the row in its array
  __device__ __forceinline__ RowWords(int h, int row)
      : H(h), start(static_cast<int64_t>(row) * h) {
    lead = ANY ? static_cast<int>(start) & 7 : 0;
  }
  // column of word v's first element (below 0 in a first word with a lead)
  __device__ __forceinline__ int column(int v) const { return 8 * v - lead; }
};
template <bool ANY>
__device__ __forceinline__ int words_of_row(int H) {
  return ANY ? (H + 14) / 8 : H / 8;  // the most that a row touches
}

// elements `col` .. `col` + 7 of an aligned row
__device__ __forceinline__ uint4 load_words(const void* array, int row, int H, int col) {
  return __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(array) +
                                               static_cast<int64_t>(row) * H + col));
}

// the word at column `col` of the row that the words were cut by
template <bool ANY>
__device__ __forceinline__ void store_words(void* array, const RowWords<ANY>& r, int col,
                                            const uint4& w) {
  uint16_t* dst = static_cast<uint16_t*>(array) + r.start + col;
  if (!ANY || (col >= 0 && col + 8 <= r.H)) {
    __stcs(reinterpret_cast<uint4*>(dst), w);
  } else {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i >= 0 && col + i < r.H)
        dst[i] = static_cast<uint16_t>(u[i / 2] >> (16 * (i & 1)));
  }
}

// ------------------------------------------------------------------ the copies
// Row x[token] to the places of its slots, by one warp: words [32 U part,
// 32 U (part + 1)) of it. `place`: the token's topk rows (below 0: dropped).
constexpr int kCopyWords = 4;  // words a lane holds (U)

template <bool ANY>
__device__ __forceinline__ void copy_item(const MoeParams& p, int token, int part,
                                          const int32_t* place) {
  constexpr int U = kCopyWords;
  const int H = p.hidden;
  const int v0 = part * (32 * U) + static_cast<int>(lane_id());
  if constexpr (!ANY) {
    const int nv = H / 8;
    const uint4* src = static_cast<const uint4*>(p.x) + static_cast<int64_t>(token) * nv + v0;
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (v0 + 32 * u < nv) v[u] = __ldcs(src + 32 * u);
    for (int s = 0; s < p.topk; ++s) {
      const int row = place[s];
      if (row < 0) continue;
      uint4* dst = static_cast<uint4*>(p.rows) + static_cast<int64_t>(row) * nv + v0;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (v0 + 32 * u < nv) __stcs(dst + 32 * u, v[u]);
    }
  } else {
    const int64_t total = 2 * static_cast<int64_t>(p.tokens) * H;
    const uint8_t* x = static_cast<const uint8_t*>(p.x);
    const bool inside = row_inside(token, p.tokens, H);
    for (int s = 0; s < p.topk; ++s) {
      const int row = place[s];
      if (row < 0) continue;
      const RowWords<true> r(H, row);
      // (the row's alignment, and so the shift, is the same for all its words)
      const int col0 = r.column(v0);
      const int64_t at0 = 2 * (static_cast<int64_t>(token) * H + col0);
      const uint32_t shift = static_cast<uint32_t>(at0) & 15u;
      uint4 a[U], b[U];
      if (inside) {
        const uint4* src = reinterpret_cast<const uint4*>(x + at0 - shift);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (col0 + 256 * u >= H) continue;
          a[u] = load_early(src + 32 * u);
          b[u] = load_early(src + 32 * u + 1);
        }
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          a[u] = word_at(x, at0 - shift + 512 * u, total);
          b[u] = word_at(x, at0 - shift + 512 * u + 16, total);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int col = col0 + 256 * u;
        if (col < H) store_words<true>(p.rows, r, col, shift_out(a[u], b[u], shift));
      }
    }
  }
}

// The same, quantised: 16 elements a lane, 8 lanes a block of 128, 512
// elements a warp.
template <typename T>
__device__ __forceinline__ void quant_item(const MoeParams& p, int token, int part,
                                           const int32_t* place) {
  const int nv = p.hidden / 16, blocks = (p.hidden + 127) / 128;
  const uint32_t lane = lane_id();
  const int v = part * 32 + static_cast<int>(lane);
  const bool in = v < nv;
  uint4 a = make_uint4(0, 0, 0, 0), b = a;
  if (in) {
    const uint4* src = static_cast<const uint4*>(p.x) + (static_cast<int64_t>(token) * nv + v) * 2;
    a = __ldcs(src);
    b = __ldcs(src + 1);
  }
  float inv;
  bool finite;
  const float sc = block_scale16<T, false>(a, b, inv, finite);
  const uint4 q = quant_words<T>(a, b, inv, finite);
  uint4* rows = static_cast<uint4*>(p.rows);
  for (int s = 0; s < p.topk; ++s) {
    const int row = place[s];
    if (row < 0 || !in) continue;
    __stcs(rows + static_cast<int64_t>(row) * nv + v, q);
    if ((lane & 7u) == 0) p.scale[static_cast<int64_t>(row) * blocks + (v >> 3)] = sc;
  }
}

template <int COPY, bool ANY>
__device__ __forceinline__ int copy_parts(int H) {
  return COPY == MOE_COPY_FP8 ? (H / 16 + 31) / 32
                              : (words_of_row<ANY>(H) + 32 * kCopyWords - 1) / (32 * kCopyWords);
}

// rows [kept, slots) of the output: zeros (e4m3: with scale 1), by thread
// `first` of `threads`
template <int COPY>
__device__ __forceinline__ void clear_tail(const MoeParams& p, int kept, int64_t first,
                                           int64_t threads) {
  const int64_t tail = p.slots - kept;
  if (tail <= 0) return;
  if constexpr (COPY == MOE_COPY_FP8) {
    const int64_t nv = p.hidden / 16, blocks = (p.hidden + 127) / 128;  // times rows: 64 bits
    uint4* zero = static_cast<uint4*>(p.rows) + kept * nv;
    for (int64_t i = first; i < tail * nv; i += threads) zero[i] = make_uint4(0, 0, 0, 0);
    float* ones = p.scale + kept * blocks;
    for (int64_t i = first; i < tail * blocks; i += threads) ones[i] = 1.0f;
  } else {
    // 16-bit zeros from element `begin` on; the array's aligned words between
    uint16_t* rows = static_cast<uint16_t*>(p.rows);
    const int64_t begin = static_cast<int64_t>(kept) * p.hidden;
    const int64_t end = static_cast<int64_t>(p.slots) * p.hidden;
    const int64_t w0 = (begin + 7) / 8, w1 = end / 8;
    for (int64_t i = w0 + first; i < w1; i += threads)
      reinterpret_cast<uint4*>(rows)[i] = make_uint4(0, 0, 0, 0);
    for (int64_t i = begin + first; i < min(8 * w0, end); i += threads) rows[i] = 0;
    for (int64_t i = max(8 * w1, begin) + first; i < end; i += threads) rows[i] = 0;
  }
}

// The copies on their own, after the sort of many slots: a warp per item, a CTA
// per 8 items, so that the hardware balances them over the SMs.
template <typename T, int COPY, bool ANY>
__global__ void __launch_bounds__(256) moe_copy_kernel(const MoeParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const int parts = copy_parts<COPY, ANY>(p.hidden);
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (item < static_cast<int64_t>(p.tokens) * parts) {
    const int token = static_cast<int>(item / parts);
    const int part = static_cast<int>(item - static_cast<int64_t>(token) * parts);
    const int32_t* place = p.row_of + static_cast<int64_t>(token) * p.topk;
    if constexpr (COPY == MOE_COPY_FP8)
      quant_item<T>(p, token, part, place);
    else
      copy_item<ANY>(p, token, part, place);
  }
  clear_tail<COPY>(p, p.offsets[p.experts], static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x,
                   static_cast<int64_t>(gridDim.x) * 256);
}

// The rows of x that this chunk's tokens are copied from, on their way to L2
// while the sort, which leaves HBM idle, ends: where x fills at most half of L2.
// Asked for before the counts have been shared they hold those up. 2048 tokens,
// 8 slots, 5120 columns: 35.4 us (e4m3 23.3), without 37.6 (24.6); 4096 tokens
// 64.4 (40.2) and 65.5 (40.7).
constexpr int64_t kPrefetchBytes = 64 << 20;

__device__ __forceinline__ void prefetch_rows(const MoeParams& p) {
  const int64_t row = 2 * static_cast<int64_t>(p.hidden), total = p.tokens * row;
  if (p.x == nullptr || total > kPrefetchBytes) return;
  // (whole 16-byte words: of an odd row's last one the copy loads the rest itself)
  const int64_t begin = min(blockIdx.x * p.chunk_tokens * row, total) & ~int64_t(15);
  const int64_t end = min((blockIdx.x + int64_t(1)) * p.chunk_tokens * row, total) & ~int64_t(15);
  constexpr int64_t kPiece = 16384;
  for (int64_t at = begin; at < end; at += kPiece)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                     static_cast<const uint8_t*>(p.x) + at),
                 "r"(static_cast<uint32_t>(min(kPiece, end - at)))
                 : "memory");
}

// The sort, and where little is copied (fused) the copies of the chunk's tokens too.
template <typename T, int COPY, bool ANY>
__global__ void __launch_bounds__(kSortThreads) moe_dispatch_kernel(const MoeParams p) {
  extern __shared__ int32_t smem[];
  int32_t* total = smem;                                // [experts], less `before`
  int32_t* before = total + p.experts;                  // [experts]
  int32_t* mine = before + p.experts;                   // [experts], of this chunk
  int32_t* rank = mine + p.experts;                     // [kRankWarps][experts]
  int32_t* place = rank + kRankWarps * p.experts;       // [chunk slots] (with copies)
  __shared__ int32_t warp_sum[kSortThreads / 32];
  static_assert(kSortThreads >= kMaxExperts, "a thread per expert");
  const int tid = threadIdx.x, warp = tid >> 5;
  const uint32_t lane = lane_id();
  const int experts = p.experts;
  const int64_t chunk_slots = static_cast<int64_t>(p.chunk_tokens) * p.topk;
  const int first = static_cast<int>(min(static_cast<int64_t>(p.slots), blockIdx.x * chunk_slots));
  const int last = static_cast<int>(min(static_cast<int64_t>(p.slots), first + chunk_slots));
  const int n = last - first;
  const bool writer = blockIdx.y == 0;  // of the chunk's CTAs, the one that writes the indexes
  // this CTA's place in its cluster, and the first slot of the cluster's chunks
  const uint32_t cta = p.clusters ? cluster_ctarank() : 0u;
  const uint32_t ctas = p.clusters ? kSortCluster : 1u;
  const int lead = static_cast<int>(
      min(static_cast<int64_t>(p.slots), (blockIdx.x - cta) * chunk_slots));

  for (int i = tid; i < (3 + kRankWarps) * experts; i += kSortThreads) smem[i] = 0;
  grid_dep_wait();
  grid_dep_launch();
  __syncthreads();

  // this CTA's part of all slots, four at a time: `before` counts what lies
  // before the cluster's chunks, `total` the rest
  const int64_t quads = (static_cast<int64_t>(p.slots) + 3) / 4;
  for (int64_t i = quads * cta / ctas + tid; i < quads * (cta + 1) / ctas; i += kSortThreads) {
    const int64_t at = 4 * i;
    int e[4];
    if (at + 4 <= p.slots) {
      const int4 v = *reinterpret_cast<const int4*>(p.expert + at);
      e[0] = v.x, e[1] = v.y, e[2] = v.z, e[3] = v.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) e[j] = at + j < p.slots ? p.expert[at + j] : -1;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (static_cast<uint32_t>(e[j]) < static_cast<uint32_t>(experts))
        atomicAdd(at + j < lead ? &before[e[j]] : &total[e[j]], 1);
  }
  // this chunk's slots of every expert, for each ranking warp's run of slots
  const int run = (n + kRankWarps * 32 - 1) / (kRankWarps * 32) * 32;
  if (warp < kRankWarps) {
    for (int i = warp * run + static_cast<int>(lane); i < min(n, (warp + 1) * run); i += 32) {
      const uint32_t e = static_cast<uint32_t>(p.expert[first + i]);
      if (e < static_cast<uint32_t>(experts)) atomicAdd(&rank[warp * experts + e], 1);
    }
  }
  __syncthreads();

  // thread t's expert: all its slots, and those before this chunk
  int all = 0, prior = 0;
  if (p.clusters) {
    if (tid < experts) {
      int sum = 0;
#pragma unroll
      for (int w = 0; w < kRankWarps; ++w) sum += rank[w * experts + tid];
      mine[tid] = sum;
    }
    __syncwarp();
    cluster_sync();
    if (tid < experts) {
#pragma unroll
      for (uint32_t c = 0; c < kSortCluster; ++c) {
        const int b = ld_cluster(mapa_shared(smem_u32(&before[tid]), c));
        all += b + ld_cluster(mapa_shared(smem_u32(&total[tid]), c));
        prior += b + (c < cta ? ld_cluster(mapa_shared(smem_u32(&mine[tid]), c)) : 0);
      }
    }
    // (no CTA ends before the others have read its counts: awaited at the end)
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  } else if (tid < experts) {
    prior = before[tid];
    all = prior + total[tid];
  }

  if (COPY == MOE_SORT_ONLY && tid == kSortThreads - 1) prefetch_rows(p);

  // the experts' first rows (exclusive sum)
  int incl = all;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (static_cast<int>(lane) >= d) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int at = incl - all;
  int kept = 0;
#pragma unroll
  for (int w = 0; w < kSortThreads / 32; ++w) {
    at += w < warp ? warp_sum[w] : 0;
    kept += warp_sum[w];
  }
  const bool index_writer = writer && blockIdx.x == 0;
  if (index_writer && tid == 0) p.offsets[experts] = kept;
  if (tid < experts) {
    if (index_writer) p.offsets[tid] = at;
    // the first row of each ranking warp's slots of this expert
    int next = at + prior;
#pragma unroll
    for (int w = 0; w < kRankWarps; ++w) {
      const int v = rank[w * experts + tid];
      rank[w * experts + tid] = next;
      next += v;
    }
  }
  __syncthreads();

  if (warp < kRankWarps) {
    for (int i0 = warp * run; i0 < min(n, (warp + 1) * run); i0 += 32) {
      const int i = i0 + static_cast<int>(lane);
      int e = -1;
      if (i < n) e = p.expert[first + i];
      if (e < 0 || e >= experts) e = -1;
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
      int row = -1;
      if (e >= 0) row = rank[warp * experts + e] + __popc(same & ((1u << lane) - 1u));
      __syncwarp();
      if (e >= 0 && static_cast<int>(lane) == __ffs(same) - 1)
        rank[warp * experts + e] += __popc(same);
      __syncwarp();
      if (i < n) {
        if constexpr (COPY != MOE_SORT_ONLY) place[i] = row;
        if (writer) {
          p.row_of[first + i] = row;
          if (row >= 0) p.slot_of[row] = first + i;
        }
      }
    }
  }
  // rows without a slot
  if (writer)
    for (int64_t r = kept + static_cast<int64_t>(blockIdx.x) * kSortThreads + tid; r < p.slots;
         r += static_cast<int64_t>(gridDim.x) * kSortThreads)  // passes 2^31 with many slots
      p.slot_of[r] = -1;
  if (p.clusters) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  if constexpr (COPY == MOE_SORT_ONLY) return;
  __syncthreads();

  const int parts = copy_parts<COPY, ANY>(p.hidden);
  const int64_t items = static_cast<int64_t>(n / p.topk) * parts;
  constexpr int kWarps = kSortThreads / 32;
  // (the first pieces to every one of the chunk's CTAs, then the next)
  for (int64_t it = static_cast<int64_t>(warp) * gridDim.y + blockIdx.y; it < items;
       it += static_cast<int64_t>(gridDim.y) * kWarps) {
    const int t = static_cast<int>(it / parts);
    const int part = static_cast<int>(it - static_cast<int64_t>(t) * parts);
    const int token = static_cast<int>(blockIdx.x) * p.chunk_tokens + t;
    if constexpr (COPY == MOE_COPY_FP8)
      quant_item<T>(p, token, part, place + t * p.topk);
    else
      copy_item<ANY>(p, token, part, place + t * p.topk);
  }
  clear_tail<COPY>(p, kept,
                   static_cast<int64_t>(blockIdx.x * gridDim.y + blockIdx.y) * kSortThreads + tid,
                   static_cast<int64_t>(gridDim.x) * gridDim.y * kSortThreads);
}

// ---------------------------------------------------------------- back again
// The slots whose loads are in flight together (KS) are a template parameter: the
// smallest of 2, 4, 6 and 8 that holds topk, 8 for more. With 8 for 2 slots the
// registers for the others cost half of the bandwidth (116 against 65 us, 16384
// tokens of 4096), with 8 for 6 a tenth (29.6 against 27.1 us, 5003 of 2047).

// out[t] = sum_s w[t][s] rows[row_of[t][s]] (WEIGHTED) or the plain sum.
template <typename T>
__device__ __forceinline__ void add_word(float2 (&acc)[4], const uint4& w, float weight) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) add_scaled(acc[i], Pair16<T>::unpack(u[i]), weight);
}

template <typename T>
__device__ __forceinline__ uint4 pack_word(const float2 (&acc)[4]) {
  return make_uint4(Pair16<T>::pack(acc[0].x, acc[0].y), Pair16<T>::pack(acc[1].x, acc[1].y),
                    Pair16<T>::pack(acc[2].x, acc[2].y), Pair16<T>::pack(acc[3].x, acc[3].y));
}

// the rows of slots s0 .. s0 + KS - 1 of token t (below 0: none)
template <int KS>
__device__ __forceinline__ void rows_of(const GatherParams& p, int t, int s0, int (&row)[KS]) {
  const int32_t* row_of = p.row_of + static_cast<int64_t>(t) * p.topk + s0;
#pragma unroll
  for (int j = 0; j < KS; ++j) {
    row[j] = s0 + j < p.topk ? row_of[j] : -1;
    if (row[j] >= p.slots) row[j] = -1;
  }
}

// their weights. KEPT: of the slots with a row only, so that the loads follow
// the rows' indexes: where the indexes are a thread's own, loads for all slots
// beside those of the rows cost 2 us of 180; where they are the CTA's, 2 of 30
// are gained.
template <bool WEIGHTED, bool KEPT, int KS>
__device__ __forceinline__ void weights_of(const GatherParams& p, int t, int s0,
                                           const int (&row)[KS], float (&weight)[KS]) {
  const float* w = p.weight + static_cast<int64_t>(t) * p.topk + s0;
#pragma unroll
  for (int j = 0; j < KS; ++j)
    weight[j] = WEIGHTED && (KEPT ? row[j] >= 0 : s0 + j < p.topk) ? w[j] : 1.0f;
}

// Aligned rows: a thread has one word of a token's row.
template <typename T, bool WEIGHTED, int KS>
__global__ void __launch_bounds__(256, 3) moe_gather_kernel(const GatherParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const int H = p.hidden, nv = H / 8;
  const int64_t items = static_cast<int64_t>(p.tokens) * nv;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; it < items;
       it += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int t = static_cast<int>(it / nv);
    const int col = 8 * static_cast<int>(it - static_cast<int64_t>(t) * nv);
    float2 acc[4] = {};
    for (int s0 = 0; s0 < p.topk; s0 += KS) {
      uint4 w[KS];
      float weight[KS];
      int row[KS];
      rows_of<KS>(p, t, s0, row);
      weights_of<WEIGHTED, true, KS>(p, t, s0, row, weight);
#pragma unroll
      for (int j = 0; j < KS; ++j)
        if (row[j] >= 0) w[j] = load_words(p.rows, row[j], H, col);
#pragma unroll
      for (int j = 0; j < KS; ++j)
        if (row[j] >= 0) add_word<T>(acc, w[j], weight[j]);
    }
    store_words<false>(p.out, RowWords<false>(H, t), col, pack_word<T>(acc));
  }
}

// Rows of any length: a CTA per token, so that the slots' rows and shifts are
// the CTA's, and a warp for 31 words at a time: its lanes load 32 aligned words
// of each row, and every lane shifts its word out of its own and the next
// lane's. (With the words of all tokens dealt out to the warps in one row the
// index arithmetic took most of the instructions: gradient of dispatch, 5003
// tokens, 6 slots, 2047 columns of fp16, 39 against 27 us.) Up to four warps a
// CTA, as few as the same number of turns needs: 27 us, with up to eight 27.5,
// with two 31. Seven CTAs' registers (72 a thread): 2000 tokens, 8 slots, 7169
// columns 47 us, with 80 registers 55.
constexpr int kAnyWarps = 4;

template <typename T, bool WEIGHTED, int KS>
__global__ void __launch_bounds__(32 * kAnyWarps, 7)
    moe_gather_any_kernel(const GatherParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const int H = p.hidden, t = static_cast<int>(blockIdx.x);
  const uint8_t* rows = static_cast<const uint8_t*>(p.rows);
  const int lane = static_cast<int>(lane_id());
  const RowWords<true> r(H, t);
  const int words = (r.lead + H + 7) / 8;
  for (int v = static_cast<int>(threadIdx.x >> 5) * 31; v < words;
       v += static_cast<int>(blockDim.x >> 5) * 31) {
    const int col = r.column(v + lane);
    float2 acc[4] = {};
    for (int s0 = 0; s0 < p.topk; s0 += KS) {
      uint4 w[KS];
      float weight[KS];
      int row[KS];
      rows_of<KS>(p, t, s0, row);
      weights_of<WEIGHTED, false, KS>(p, t, s0, row, weight);
      bool inside = true;
#pragma unroll
      for (int j = 0; j < KS; ++j)
        inside = inside && (row[j] < 0 || row_inside(row[j], p.slots, H));
      // (a lane up to one word past the row still loads for the one before it)
      if (inside) {
#pragma unroll
        for (int j = 0; j < KS; ++j)
          if (row[j] >= 0 && col < H + 8)
            w[j] = __ldcs(reinterpret_cast<const uint4*>(
                rows + (2 * (static_cast<int64_t>(row[j]) * H + col) & ~int64_t(15))));
      } else {
        const int64_t total = 2 * static_cast<int64_t>(p.slots) * H;
#pragma unroll
        for (int j = 0; j < KS; ++j)
          if (row[j] >= 0 && col < H + 8)
            w[j] = word_at(rows, 2 * (static_cast<int64_t>(row[j]) * H + col) & ~int64_t(15),
                           total);
      }
      __syncwarp();
#pragma unroll
      for (int j = 0; j < KS; ++j)
        if (row[j] >= 0)  // the same in the whole CTA, and so the shift: column() is -lead mod 8
          add_word<T>(acc,
                      shift_in(w[j], 2 * (static_cast<uint32_t>(row[j]) * H -
                                          static_cast<uint32_t>(r.lead)) & 15u),
                      weight[j]);
    }
    if (lane < 31 && col < H) store_words<true>(p.out, r, col, pack_word<T>(acc));
  }
}

// d_rows[row] = w d_out[t], d_weight[t][s] = <d_out[t], rows[row]>: a CTA per
// token. A thread adds its words' products per slot, the warps' sums are added
// in a fixed order.
constexpr int kGradWarps = 4;  // most of a CTA
// The words of all slots at once are in flight, and as many CTAs as the
// registers for them allow: 5003 tokens, 6 slots, 2047 columns 58 us, with one
// word in flight 70, with the compiler's own number of registers 66; 16384
// tokens, 8 slots, 4096 columns 337, 340 without the bound.
constexpr int grad_ctas(int slots) { return slots == 8 ? 5 : slots == 6 ? 7 : slots == 4 ? 9 : 12; }

// one word of a slot: dot += <d, x>, and w d
template <typename T>
__device__ __forceinline__ uint4 grad_word(float2& dot, const uint4& d, const uint4& x, float w) {
  const uint32_t du[4] = {d.x, d.y, d.z, d.w}, xu[4] = {x.x, x.y, x.z, x.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = Pair16<T>::unpack(du[i]);
    const float2 g = Pair16<T>::unpack(xu[i]);
    dot.x = fmaf(f.x, g.x, dot.x);
    dot.y = fmaf(f.y, g.y, dot.y);
    o[i] = Pair16<T>::pack(f.x * w, f.y * w);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// the word's elements of columns outside [0, H) (a neighbour's) set to zero
__device__ __forceinline__ uint4 inside_row(const uint4& x, int col, int H) {
  uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = col + 2 * i;
    u[i] &= (c >= 0 && c < H ? 0xFFFFu : 0u) | (c + 1 >= 0 && c + 1 < H ? 0xFFFF0000u : 0u);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

template <typename T, bool ANY, int KS>
__global__ void __launch_bounds__(32 * kGradWarps, grad_ctas(KS))
    moe_combine_grad_kernel(const GatherParams p) {
  __shared__ float part[64][kGradWarps];
  grid_dep_wait();
  grid_dep_launch();
  const int H = p.hidden, nv = words_of_row<ANY>(H);
  const int t = static_cast<int>(blockIdx.x);
  const int64_t slot0 = static_cast<int64_t>(t) * p.topk;
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t total = 2 * static_cast<int64_t>(p.tokens) * H;
  const int64_t total_rows = 2 * static_cast<int64_t>(p.slots) * H;
  const uint8_t* rows = static_cast<const uint8_t*>(p.rows);
  const uint8_t* d_out = static_cast<const uint8_t*>(p.d_out);
  const int64_t d_start = static_cast<int64_t>(t) * H;
  for (int s0 = 0; s0 < p.topk; s0 += KS) {
    float2 dot[KS] = {};
    float w[KS];
    int row[KS];
    bool inside = ANY && row_inside(t, p.tokens, H);
    rows_of<KS>(p, t, s0, row);
    weights_of<true, false, KS>(p, t, s0, row, w);
#pragma unroll
    for (int j = 0; j < KS; ++j)
      if (ANY) inside = inside && (row[j] < 0 || row_inside(row[j], p.slots, H));
    for (int v = threadIdx.x; v < nv; v += blockDim.x) {
      uint4 x[KS];
      if constexpr (!ANY) {
        const uint4 d = *reinterpret_cast<const uint4*>(d_out + 2 * (d_start + 8 * v));
#pragma unroll
        for (int j = 0; j < KS; ++j)
          if (row[j] >= 0) x[j] = load_words(p.rows, row[j], H, 8 * v);
#pragma unroll
        for (int j = 0; j < KS; ++j)
          if (row[j] >= 0)
            store_words<false>(p.out, RowWords<false>(H, row[j]), 8 * v,
                               grad_word<T>(dot[j], d, x[j], w[j]));
      } else {
        // the words of rows and d_rows, which start alike, differ from slot to
        // slot, and so does what they need of d_out
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          if (row[j] < 0) continue;
          const RowWords<true> r(H, row[j]);
          const int64_t at = 2 * (r.start + r.column(v));
          if (r.column(v) < H)
            x[j] = inside ? __ldcs(reinterpret_cast<const uint4*>(rows + at))
                          : word_at(rows, at, total_rows);
        }
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          if (row[j] < 0) continue;
          const RowWords<true> r(H, row[j]);
          const int col = r.column(v);
          if (col >= H) continue;
          const int64_t at = 2 * (d_start + col);
          uint4 d;
          if (inside) {
            const uint32_t shift = static_cast<uint32_t>(at) & 15u;
            const uint4* src = reinterpret_cast<const uint4*>(d_out + at - shift);
            d = shift_out(load_early(src), load_early(src + 1), shift);
          } else {
            d = bytes_at(d_out, at, total);
          }
          if (col < 0 || col + 8 > H) {
            d = inside_row(d, col, H);
            x[j] = inside_row(x[j], col, H);
          }
          store_words<true>(p.out, r, col, grad_word<T>(dot[j], d, x[j], w[j]));
        }
      }
    }
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      float sum = dot[j].x + dot[j].y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      if (lane_id() == 0 && s0 + j < p.topk) part[s0 + j][warp] = sum;
    }
  }
  __syncthreads();
  for (int s = threadIdx.x; s < p.topk; s += blockDim.x) {
    float dot = 0.0f;
    for (int i = 0; i < warps; ++i) dot += part[s][i];
    p.d_weight[slot0 + s] = dot;
  }
  // rows without a slot
  MoeParams tail = {};
  tail.slots = p.slots;
  tail.hidden = H;
  tail.rows = p.out;
  clear_tail<MOE_COPY>(tail, min(max(p.offsets[p.experts], 0), p.slots),
                       static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x,
                       static_cast<int64_t>(gridDim.x) * blockDim.x);
}

// -------------------------------------------------------------- quantisation
// 1 x 128 blocks: 16 elements a lane, 8 lanes a block. A thread has two such
// runs, 256 apart, both in flight.
template <typename T>
__global__ void __launch_bounds__(256) quantize_rows_kernel(int64_t m, int64_t k, const uint4* x,
                                                            uint4* q, float* scale) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t nv = k / 16, blocks = (k + 127) / 128;
  const int64_t padded = blocks * 8;  // lanes of a row, whole blocks
  const int64_t items = m * padded;
  // (items is a multiple of 8: the shuffles stay in a block)
  const int64_t first = static_cast<int64_t>(blockIdx.x) * 512 + threadIdx.x;
  uint4 a[2], b[2];
  int64_t r[2], v[2];
  bool in[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t it = first + 256 * i;
    r[i] = it / padded;
    v[i] = it - r[i] * padded;
    in[i] = it < items && v[i] < nv;
    a[i] = make_uint4(0, 0, 0, 0);
    b[i] = a[i];
    if (in[i]) {
      a[i] = __ldcs(x + (r[i] * nv + v[i]) * 2);
      b[i] = __ldcs(x + (r[i] * nv + v[i]) * 2 + 1);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float inv;
    bool finite;
    const float sc = block_scale16<T, true>(a[i], b[i], inv, finite);
    if (in[i]) {
      __stcs(q + r[i] * nv + v[i], quant_words<T>(a[i], b[i], inv, finite));
      if ((v[i] & 7) == 0) scale[r[i] * blocks + (v[i] >> 3)] = sc;
    }
  }
}

// 128 x 128 blocks: a CTA per block, its elements held in registers between
// the maximum and the rounding; three CTAs an SM keep loads in flight while
// others convert (17408 x 5120 bf16: 42.2 us; four CTAs 47, two 50, six of 256
// threads 49, 8 elements a lane with 8-byte stores 44; with the maximum taken of
// floats instead of 16-bit pairs 45.2).
constexpr int kBlockThreads = 512;

template <typename T>
__global__ void __launch_bounds__(kBlockThreads, 3)
    quantize_blocks_kernel(int64_t m, int64_t k, int blocks_k, const uint4* x, uint4* q,
                           float* scale) {
  __shared__ uint32_t warp_mag[kBlockThreads / 32];
  grid_dep_wait();
  grid_dep_launch();
  const int64_t nv = k / 16;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x / blocks_k) * 128 + (threadIdx.x >> 3);
  const int64_t v = static_cast<int64_t>(blockIdx.x % blocks_k) * 8 + (threadIdx.x & 7);
  uint4 a[2], b[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t r = r0 + (kBlockThreads / 8) * i;
    a[i] = make_uint4(0, 0, 0, 0);
    b[i] = a[i];
    if (r < m && v < nv) {
      a[i] = __ldcs(x + (r * nv + v) * 2);
      b[i] = __ldcs(x + (r * nv + v) * 2 + 1);
    }
  }
  // the block's largest magnitude; with an infinity or NaN in it once more,
  // without those
  auto largest = [&](uint32_t mag2) {
    const uint32_t own = __reduce_max_sync(0xFFFFFFFFu, fold2(mag2));
    if ((threadIdx.x & 31) == 0) warp_mag[threadIdx.x >> 5] = own;
    __syncthreads();
    uint32_t mag = 0;
#pragma unroll
    for (int w = 0; w < kBlockThreads / 32; ++w) mag = max(mag, warp_mag[w]);
    return mag;
  };
  uint32_t mag2 = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) mag2 = max_mag2<T>(max_mag2<T>(mag2, a[i]), b[i]);
  uint32_t mag = largest(mag2);
  const bool finite = mag < kInf16<T>;
  if (!finite) {
    mag2 = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      mag2 = max_mag2<T, true>(max_mag2<T, true>(mag2, a[i]), b[i]);
    __syncthreads();  // all have read the first maxima
    mag = largest(mag2);
  }
  float inv;
  const float sc = e4m3_scale(mag_to_f32<T>(mag), inv);
  if (threadIdx.x == 0) scale[blockIdx.x] = sc;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t r = r0 + (kBlockThreads / 8) * i;
    if (r < m && v < nv) __stcs(q + r * nv + v, quant_words<T>(a[i], b[i], inv, finite));
  }
}

template <typename T>
cudaError_t dispatch_t(const MoeParams& p, int copy, cudaStream_t stream, int pdl) {
  const bool any = p.hidden % 8 != 0;
  // little to copy: the sort and the copies in one kernel
  const int fused = p.fused ? copy : MOE_SORT_ONLY;
  const unsigned cluster = p.clusters ? kSortCluster : 1;
  const dim3 grid((p.num_chunks + cluster - 1) / cluster * cluster,
                  fused == MOE_SORT_ONLY ? 1 : p.segments, 1);
  const size_t places = fused == MOE_SORT_ONLY ? 0 : size_t(p.chunk_tokens) * p.topk;
  const size_t smem = ((3 + kRankWarps) * static_cast<size_t>(p.experts) + places) * 4;
  // Without asking, a kernel has 48 KB, its static arrays among them (below 1 KB
  // here). The limit is the kernel's, not the launch's: always raised to the most
  // that any plan takes, so that no call lowers it between another's two steps.
  constexpr int kMostSmem = ((3 + kRankWarps) * kMaxExperts + kMoeChunkSlots) * 4;
  auto sort = [&](auto kernel) -> cudaError_t {
    if (smem > 47 * 1024) {
      const cudaError_t e = cudaFuncSetAttribute(
          kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
      if (e != cudaSuccess) return e;
    }
    return launch_clusters(kernel, grid, cluster, kSortThreads, smem, stream, pdl, p);
  };
  const cudaError_t e =
      fused == MOE_SORT_ONLY  ? sort(moe_dispatch_kernel<T, MOE_SORT_ONLY, false>)
      : fused == MOE_COPY_FP8 ? sort(moe_dispatch_kernel<T, MOE_COPY_FP8, false>)
      : any                   ? sort(moe_dispatch_kernel<T, MOE_COPY, true>)
                              : sort(moe_dispatch_kernel<T, MOE_COPY, false>);
  if (e != cudaSuccess || fused == copy) return e;
  const int64_t parts = copy == MOE_COPY_FP8 ? (p.hidden / 16 + 31) / 32
                        : any ? ((p.hidden + 14) / 8 + 32 * kCopyWords - 1) / (32 * kCopyWords)
                              : (p.hidden / 8 + 32 * kCopyWords - 1) / (32 * kCopyWords);
  auto go = [&](auto kernel) {
    return launch(kernel, dim3(static_cast<unsigned>((p.tokens * parts + 7) / 8)), 256, 0, stream,
                  pdl, p);
  };
  return copy == MOE_COPY_FP8 ? go(moe_copy_kernel<T, MOE_COPY_FP8, false>)
         : any                ? go(moe_copy_kernel<T, MOE_COPY, true>)
                              : go(moe_copy_kernel<T, MOE_COPY, false>);
}

// calls f with the number of slots at once
template <typename F>
cudaError_t for_slots(int topk, F f) {
  if (topk <= 2) return f(std::integral_constant<int, 2>());
  if (topk <= 4) return f(std::integral_constant<int, 4>());
  if (topk <= 6) return f(std::integral_constant<int, 6>());
  return f(std::integral_constant<int, 8>());
}

// up to `most` warps for `windows` of a row: as few as the same turns need
int even_warps(int windows, int most) {
  const int turns = (windows + most - 1) / most;
  return turns == 0 ? 1 : (windows + turns - 1) / turns;
}

template <typename T>
cudaError_t gather_t(const GatherParams& p, int sms, cudaStream_t stream, int pdl) {
  if (p.hidden % 8 != 0) {
    const int threads = 32 * even_warps(((p.hidden + 14) / 8 + 30) / 31, kAnyWarps);
    return for_slots(p.topk, [&](auto ks) {
      constexpr int KS = decltype(ks)::value;
      auto go = [&](auto kernel) {
        return launch(kernel, dim3(static_cast<unsigned>(p.tokens)), threads, 0, stream, pdl, p);
      };
      return p.weight ? go(moe_gather_any_kernel<T, true, KS>)
                      : go(moe_gather_any_kernel<T, false, KS>);
    });
  }
  const int64_t items = static_cast<int64_t>(p.tokens) * (p.hidden / 8);
  const int64_t want = (items + 255) / 256, most = static_cast<int64_t>(sms) * 64;
  const dim3 grid(static_cast<unsigned>(want < most ? want : most));
  return for_slots(p.topk, [&](auto ks) {
    constexpr int KS = decltype(ks)::value;
    auto go = [&](auto kernel) { return launch(kernel, grid, 256, 0, stream, pdl, p); };
    return p.weight ? go(moe_gather_kernel<T, true, KS>) : go(moe_gather_kernel<T, false, KS>);
  });
}

template <typename T>
cudaError_t grad_t(const GatherParams& p, cudaStream_t stream, int pdl) {
  const dim3 grid(static_cast<unsigned>(p.tokens));
  const bool any = p.hidden % 8 != 0;
  const int threads =
      32 * even_warps(((any ? p.hidden + 14 : p.hidden) / 8 + 31) / 32, kGradWarps);
  return for_slots(p.topk, [&](auto ks) {
    constexpr int KS = decltype(ks)::value;
    auto go = [&](auto kernel) { return launch(kernel, grid, threads, 0, stream, pdl, p); };
    return any ? go(moe_combine_grad_kernel<T, true, KS>)
               : go(moe_combine_grad_kernel<T, false, KS>);
  });
}

}  // namespace

cudaError_t launch_moe_dispatch(const MoeParams& p, int copy, int bf16, cudaStream_t stream,
                                int pdl) {
  return bf16 ? dispatch_t<__nv_bfloat16>(p, copy, stream, pdl)
              : dispatch_t<__half>(p, copy, stream, pdl);
}

cudaError_t launch_moe_gather(const GatherParams& p, int bf16, int sms, cudaStream_t stream,
                              int pdl) {
  return bf16 ? gather_t<__nv_bfloat16>(p, sms, stream, pdl)
              : gather_t<__half>(p, sms, stream, pdl);
}

cudaError_t launch_moe_combine_grad(const GatherParams& p, int bf16, cudaStream_t stream,
                                    int pdl) {
  return bf16 ? grad_t<__nv_bfloat16>(p, stream, pdl) : grad_t<__half>(p, stream, pdl);
}

cudaError_t launch_fp8_quantize(int64_t m, int64_t k, int bf16, int block_rows, const void* x,
                                void* q, float* scale, cudaStream_t stream, int pdl) {
  const uint4* src = static_cast<const uint4*>(x);
  uint4* dst = static_cast<uint4*>(q);
  const int64_t blocks_k = (k + 127) / 128;
  if (block_rows == 128) {
    const dim3 grid(static_cast<unsigned>((m + 127) / 128 * blocks_k));
    auto go = [&](auto kernel) {
      return launch(kernel, grid, kBlockThreads, 0, stream, pdl, m, k, static_cast<int>(blocks_k),
                    src, dst, scale);
    };
    return bf16 ? go(quantize_blocks_kernel<__nv_bfloat16>) : go(quantize_blocks_kernel<__half>);
  }
  const dim3 grid(static_cast<unsigned>((m * blocks_k * 8 + 511) / 512));
  auto go = [&](auto kernel) {
    return launch(kernel, grid, 256, 0, stream, pdl, m, k, src, dst, scale);
  };
  return bf16 ? go(quantize_rows_kernel<__nv_bfloat16>) : go(quantize_rows_kernel<__half>);
}

}  // namespace gf
