// Expert routing: the stable sort of the (token, slot) pairs by expert, the
// copies of the tokens' rows to their places and back, and their gradients.
//
// Everything here is bound by HBM: the arithmetic is a few operations per
// element. Each kernel is token-driven, so that the one row that all of a
// token's slots share (x, out, d_out) passes through the chip once and only
// the topk rows per token that differ are read or written.
#include <type_traits>

#include "fp8.cuh"
#include "moe.h"
#include "ptx.cuh"

namespace gf {
namespace {

constexpr int kSortThreads = 512;
constexpr int kRankWarps = 8;        // warps that rank the slots of a chunk
constexpr int kMaxChunkSlots = 4096;

template <typename K, typename... A>
cudaError_t launch(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, int pdl,
                   A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ------------------------------------------------------------------- the sort
// A counting sort over chunks of consecutive tokens, one CTA each: the place
// of a slot is its expert's first row, plus the kept slots of that expert in
// earlier chunks, in earlier warps of its chunk and earlier in its warp. Every
// term is a count, so the order is stable and the same in every run.

// counts[chunk][e]: the chunk's slots of expert e
__global__ void __launch_bounds__(kSortThreads) moe_count_kernel(const MoeParams p) {
  extern __shared__ int32_t hist[];
  grid_dep_wait();
  grid_dep_launch();
  for (int e = threadIdx.x; e < p.experts; e += kSortThreads) hist[e] = 0;
  __syncthreads();
  const int first = blockIdx.x * p.chunk_tokens * p.topk;
  const int last = min(p.slots, first + p.chunk_tokens * p.topk);
  for (int i = first + threadIdx.x; i < last; i += kSortThreads) {
    const uint32_t e = static_cast<uint32_t>(p.expert[i]);
    if (e < static_cast<uint32_t>(p.experts)) atomicAdd(&hist[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.experts; e += kSortThreads)
    p.counts[static_cast<int64_t>(blockIdx.x) * p.experts + e] = hist[e];
}

// one 16-byte or 2-byte element of a row
template <int VEC>
struct Elem {
  using type = typename std::conditional<VEC == 8, uint4, uint16_t>::type;
};

// VEC: elements per access, 8 where rows are multiples of 16 bytes, else 1.
template <typename T, int COPY, int VEC>
__global__ void __launch_bounds__(kSortThreads) moe_dispatch_kernel(const MoeParams p) {
  extern __shared__ int32_t smem[];
  int32_t* total = smem;                                // [experts]
  int32_t* before = total + p.experts;                  // [experts]
  int32_t* rank = before + p.experts;                   // [kRankWarps][experts]
  int32_t* place = rank + kRankWarps * p.experts;       // [chunk slots]
  __shared__ int32_t warp_sum[kSortThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5;
  const uint32_t lane = lane_id();
  const int experts = p.experts;
  const int first = blockIdx.x * p.chunk_tokens * p.topk;
  const int last = min(p.slots, first + p.chunk_tokens * p.topk);
  const int n = last - first;
  const bool writer = blockIdx.y == 0;  // of the chunk's CTAs, the one that writes the indexes

  for (int i = tid; i < (2 + kRankWarps) * experts; i += kSortThreads) smem[i] = 0;
  grid_dep_wait();
  grid_dep_launch();
  __syncthreads();

  // the slots of every expert: in all chunks, and in the chunks before this
  if (p.one_pass) {
    for (int i = tid; i < p.slots; i += kSortThreads) {
      const uint32_t e = static_cast<uint32_t>(p.expert[i]);
      if (e < static_cast<uint32_t>(experts)) {
        atomicAdd(&total[e], 1);
        if (i < first) atomicAdd(&before[e], 1);
      }
    }
  } else {
    // a warp's 32 lanes take 32 experts, the warps different chunks
    for (int e0 = 0; e0 < experts; e0 += 32) {
      const int e = e0 + static_cast<int>(lane);
      if (e >= experts) continue;
      int all = 0, prior = 0;
      for (int c = warp; c < p.num_chunks; c += kSortThreads / 32) {
        const int v = p.counts[static_cast<int64_t>(c) * experts + e];
        all += v;
        prior += c < static_cast<int>(blockIdx.x) ? v : 0;
      }
      atomicAdd(&total[e], all);
      atomicAdd(&before[e], prior);
    }
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

  // total -> the expert's first row (exclusive sum); thread t has the experts
  // per * t .. per * t + per - 1
  const int per = (experts + kSortThreads - 1) / kSortThreads;
  int sum = 0;
  for (int j = 0; j < per; ++j) {
    const int e = per * tid + j;
    sum += e < experts ? total[e] : 0;
  }
  int incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (static_cast<int>(lane) >= d) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int at = incl - sum;
  int kept = 0;
  for (int w = 0; w < kSortThreads / 32; ++w) {
    at += w < warp ? warp_sum[w] : 0;
    kept += warp_sum[w];
  }
  const bool index_writer = writer && blockIdx.x == 0;
  if (index_writer && tid == 0) p.offsets[experts] = kept;
  for (int j = 0; j < per; ++j) {
    const int e = per * tid + j;
    if (e >= experts) break;
    if (index_writer) p.offsets[e] = at;
    // the first row of each ranking warp's slots of this expert
    int next = at + before[e];
    for (int w = 0; w < kRankWarps; ++w) {
      const int v = rank[w * experts + e];
      rank[w * experts + e] = next;
      next += v;
    }
    at += total[e];
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
        place[i] = row;
        if (writer) {
          p.row_of[first + i] = row;
          if (row >= 0) p.slot_of[row] = first + i;
        }
      }
    }
  }
  // rows without a slot
  if (writer)
    for (int r = kept + blockIdx.x * kSortThreads + tid; r < p.slots;
         r += gridDim.x * kSortThreads)
      p.slot_of[r] = -1;
  if constexpr (COPY == MOE_SORT_ONLY) return;
  __syncthreads();

  const int64_t H = p.hidden;
  const int tokens = n / p.topk;
  const int first_token = blockIdx.x * p.chunk_tokens;
  const int cta = blockIdx.x * gridDim.y + blockIdx.y;
  const int ctas = gridDim.x * gridDim.y;
  if constexpr (COPY == MOE_COPY) {
    using V = typename Elem<VEC>::type;
    const int64_t nv = H / VEC;
    const V* x = static_cast<const V*>(p.x);
    V* rows = static_cast<V*>(p.rows);
    // a warp takes (token, run of 32 * U vectors) pairs; the CTAs of a chunk
    // take every segments-th pair
    constexpr int U = 4;
    const int parts = static_cast<int>((nv + 32 * U - 1) / (32 * U));
    const int64_t items = static_cast<int64_t>(tokens) * parts;
    for (int64_t it = static_cast<int64_t>(blockIdx.y) * (kSortThreads / 32) + warp; it < items;
         it += static_cast<int64_t>(gridDim.y) * (kSortThreads / 32)) {
      const int t = static_cast<int>(it / parts);
      const int64_t v0 = (it % parts) * (32 * U) + lane;
      V v[U];
      const V* src = x + (first_token + t) * nv;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (v0 + 32 * u < nv) v[u] = __ldcs(src + v0 + 32 * u);
      for (int s = 0; s < p.topk; ++s) {
        const int row = place[t * p.topk + s];
        if (row < 0) continue;
        V* dst = rows + static_cast<int64_t>(row) * nv;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (v0 + 32 * u < nv) __stcs(dst + v0 + 32 * u, v[u]);
      }
    }
    const int64_t tail = static_cast<int64_t>(p.slots - kept) * nv;
    V* zero = rows + static_cast<int64_t>(kept) * nv;
    for (int64_t i = static_cast<int64_t>(cta) * kSortThreads + tid; i < tail;
         i += static_cast<int64_t>(ctas) * kSortThreads)
      zero[i] = V{};
  } else {
    // 16 elements a lane, 8 lanes a block of 128, 512 elements a warp
    const int64_t nv = H / 16;
    const int blocks = static_cast<int>((H + 127) / 128);
    const uint4* x = static_cast<const uint4*>(p.x);
    uint4* rows = static_cast<uint4*>(p.rows);
    const int parts = static_cast<int>((nv + 31) / 32);
    const int64_t items = static_cast<int64_t>(tokens) * parts;
    for (int64_t it = static_cast<int64_t>(blockIdx.y) * (kSortThreads / 32) + warp; it < items;
         it += static_cast<int64_t>(gridDim.y) * (kSortThreads / 32)) {
      const int t = static_cast<int>(it / parts);
      const int64_t v = (it % parts) * 32 + lane;
      const bool in = v < nv;
      uint4 a = make_uint4(0, 0, 0, 0), b = a;
      if (in) {
        const uint4* src = x + ((first_token + t) * nv + v) * 2;
        a = __ldcs(src);
        b = __ldcs(src + 1);
      }
      float f[16];
      uint32_t mag = unpack16<T>(a, b, f);
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, d));
      float inv;
      const float sc = e4m3_scale(mag, inv);
      const uint4 q = quant16(f, inv);
      for (int s = 0; s < p.topk; ++s) {
        const int row = place[t * p.topk + s];
        if (row < 0 || !in) continue;
        rows[static_cast<int64_t>(row) * nv + v] = q;
        if ((lane & 7u) == 0) p.scale[static_cast<int64_t>(row) * blocks + (v >> 3)] = sc;
      }
    }
    const int64_t tail = static_cast<int64_t>(p.slots - kept);
    uint4* zero = rows + static_cast<int64_t>(kept) * nv;
    float* ones = p.scale + static_cast<int64_t>(kept) * blocks;
    for (int64_t i = static_cast<int64_t>(cta) * kSortThreads + tid; i < tail * nv;
         i += static_cast<int64_t>(ctas) * kSortThreads)
      zero[i] = make_uint4(0, 0, 0, 0);
    for (int64_t i = static_cast<int64_t>(cta) * kSortThreads + tid; i < tail * blocks;
         i += static_cast<int64_t>(ctas) * kSortThreads)
      ones[i] = 1.0f;
  }
}

// ---------------------------------------------------------------- back again
// Elements of a row as fp32: VEC 16-bit elements per access.
template <typename T, int VEC>
__device__ __forceinline__ void load_f32(const T* src, float (&f)[VEC]) {
  if constexpr (VEC == 8) {
    const uint4 w = __ldcs(reinterpret_cast<const uint4*>(src));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = Pair16<T>::unpack(u[i]);
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  } else {
    f[0] = Pair16<T>::one(*src);
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_f32(T* dst, const float (&f)[VEC]) {
  if constexpr (VEC == 8) {
    __stcs(reinterpret_cast<uint4*>(dst),
           make_uint4(Pair16<T>::pack(f[0], f[1]), Pair16<T>::pack(f[2], f[3]),
                      Pair16<T>::pack(f[4], f[5]), Pair16<T>::pack(f[6], f[7])));
  } else {
    *dst = Pair16<T>::round(f[0]);
  }
}

// out[t] = sum_s w[t][s] rows[row_of[t][s]] (WEIGHTED) or the plain sum. A
// thread has VEC columns of one token.
template <typename T, int VEC, bool WEIGHTED>
__global__ void __launch_bounds__(256) moe_gather_kernel(const GatherParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t nv = p.hidden / VEC;
  const T* rows = static_cast<const T*>(p.rows);
  T* out = static_cast<T*>(p.out);
  const int64_t items = p.tokens * nv;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; it < items;
       it += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t t = it / nv;
    const int64_t c = (it - t * nv) * VEC;
    float acc[VEC] = {};
    for (int s = 0; s < p.topk; ++s) {
      const int row = p.row_of[t * p.topk + s];
      if (row < 0 || row >= p.slots) continue;
      float f[VEC];
      load_f32<T, VEC>(rows + row * p.hidden + c, f);
      const float w = WEIGHTED ? p.weight[t * p.topk + s] : 1.0f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] = fmaf(w, f[i], acc[i]);
    }
    store_f32<T, VEC>(out + t * p.hidden + c, acc);
  }
}

// d_rows[row] = w d_out[t], d_weight[t][s] = <d_out[t], rows[row]>: a CTA per
// token, its threads' partial dot products added in a fixed order.
constexpr int kGradThreads = 128;

template <typename T, int VEC>
__global__ void __launch_bounds__(kGradThreads) moe_combine_grad_kernel(const GatherParams p) {
  __shared__ float part[64][kGradThreads / 32];
  grid_dep_wait();
  grid_dep_launch();
  const int64_t nv = p.hidden / VEC;
  const int warp = threadIdx.x >> 5;
  const uint32_t lane = lane_id();
  const T* rows = static_cast<const T*>(p.rows);
  T* d_rows = static_cast<T*>(p.out);
  if (static_cast<int>(blockIdx.x) < p.tokens) {
    const int64_t t = blockIdx.x;
    const T* d_out = static_cast<const T*>(p.d_out) + t * p.hidden;
    for (int s = 0; s < p.topk; ++s) {
      const int row = p.row_of[t * p.topk + s];
      float dot = 0.0f;
      if (row >= 0 && row < p.slots) {
        const float w = p.weight[t * p.topk + s];
        for (int64_t v = threadIdx.x; v < nv; v += kGradThreads) {
          float d[VEC], r[VEC];
          load_f32<T, VEC>(d_out + v * VEC, d);
          load_f32<T, VEC>(rows + row * p.hidden + v * VEC, r);
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            dot = fmaf(d[i], r[i], dot);
            d[i] *= w;
          }
          store_f32<T, VEC>(d_rows + row * p.hidden + v * VEC, d);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
      if (lane == 0) part[s][warp] = dot;
    }
    __syncthreads();
    for (int s = threadIdx.x; s < p.topk; s += kGradThreads) {
      float dot = 0.0f;
      for (int w = 0; w < kGradThreads / 32; ++w) dot += part[s][w];
      p.d_weight[t * p.topk + s] = dot;
    }
  }
  // rows without a slot
  const int kept = min(max(p.offsets[p.experts], 0), p.slots);
  const int64_t tail = static_cast<int64_t>(p.slots - kept) * nv;
  float z[VEC] = {};
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kGradThreads + threadIdx.x; i < tail;
       i += static_cast<int64_t>(gridDim.x) * kGradThreads)
    store_f32<T, VEC>(d_rows + kept * p.hidden + i * VEC, z);
}

// -------------------------------------------------------------- quantisation
// 1 x 128 blocks: 16 elements a lane, 8 lanes a block.
template <typename T>
__global__ void __launch_bounds__(256) quantize_rows_kernel(int64_t m, int64_t k, const uint4* x,
                                                            uint4* q, float* scale) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t nv = k / 16, blocks = (k + 127) / 128;
  const int64_t padded = blocks * 8;  // lanes of a row, whole blocks
  const int64_t items = m * padded;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  // whole warps go round: items is a multiple of 8, the shuffles stay in a block
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
       it - static_cast<int64_t>(lane_id()) < items; it += step) {
    const int64_t r = it / padded, v = it - r * padded;
    const bool in = it < items && v < nv;
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (in) {
      a = __ldcs(x + (r * nv + v) * 2);
      b = __ldcs(x + (r * nv + v) * 2 + 1);
    }
    float f[16];
    uint32_t mag = unpack16<T>(a, b, f);
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, d));
    float inv;
    const float sc = e4m3_scale(mag, inv);
    if (in) {
      q[r * nv + v] = quant16(f, inv);
      if ((v & 7) == 0) scale[r * blocks + (v >> 3)] = sc;
    }
  }
}

// 128 x 128 blocks: a CTA per block, its elements held in registers between
// the maximum and the rounding.
template <typename T>
__global__ void __launch_bounds__(256) quantize_blocks_kernel(int64_t m, int64_t k, int blocks_k,
                                                              const uint4* x, uint4* q,
                                                              float* scale) {
  __shared__ uint32_t warp_mag[8];
  grid_dep_wait();
  grid_dep_launch();
  const int64_t nv = k / 16;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x / blocks_k) * 128;
  const int kb = blockIdx.x % blocks_k;
  const int64_t v = static_cast<int64_t>(kb) * 8 + (threadIdx.x & 7);
  float f[4][16];
  uint32_t mag = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + 32 * i + (threadIdx.x >> 3);
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (r < m && v < nv) {
      a = __ldcs(x + (r * nv + v) * 2);
      b = __ldcs(x + (r * nv + v) * 2 + 1);
    }
    mag = max(mag, unpack16<T>(a, b, f[i]));
  }
  mag = __reduce_max_sync(0xFFFFFFFFu, mag);
  if ((threadIdx.x & 31) == 0) warp_mag[threadIdx.x >> 5] = mag;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) mag = max(mag, warp_mag[w]);
  float inv;
  const float sc = e4m3_scale(mag, inv);
  if (threadIdx.x == 0) scale[blockIdx.x] = sc;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + 32 * i + (threadIdx.x >> 3);
    if (r < m && v < nv) q[r * nv + v] = quant16(f[i], inv);
  }
}

template <typename T>
cudaError_t dispatch_t(const MoeParams& p, int copy, cudaStream_t stream, int pdl) {
  const dim3 grid(p.num_chunks, copy == MOE_SORT_ONLY ? 1 : p.segments, 1);
  const size_t smem =
      ((2 + kRankWarps) * static_cast<size_t>(p.experts) + p.chunk_tokens * p.topk) * 4;
  auto go = [&](auto kernel) -> cudaError_t {
    if (smem > 48 * 1024) {
      const cudaError_t e =
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(smem));
      if (e != cudaSuccess) return e;
    }
    return launch(kernel, grid, kSortThreads, smem, stream, pdl, p);
  };
  if (copy == MOE_SORT_ONLY) return go(moe_dispatch_kernel<T, MOE_SORT_ONLY, 1>);
  if (copy == MOE_COPY_FP8) return go(moe_dispatch_kernel<T, MOE_COPY_FP8, 8>);
  return p.hidden % 8 == 0 ? go(moe_dispatch_kernel<T, MOE_COPY, 8>)
                           : go(moe_dispatch_kernel<T, MOE_COPY, 1>);
}

}  // namespace

int moe_max_chunk_slots() { return kMaxChunkSlots; }

cudaError_t launch_moe_count(const MoeParams& p, cudaStream_t stream, int pdl) {
  return launch(moe_count_kernel, dim3(p.num_chunks), kSortThreads,
                static_cast<size_t>(p.experts) * 4, stream, pdl, p);
}

cudaError_t launch_moe_dispatch(const MoeParams& p, int copy, int bf16, cudaStream_t stream,
                                int pdl) {
  return bf16 ? dispatch_t<__nv_bfloat16>(p, copy, stream, pdl)
              : dispatch_t<__half>(p, copy, stream, pdl);
}

cudaError_t launch_moe_gather(const GatherParams& p, int bf16, int sms, cudaStream_t stream,
                              int pdl) {
  const bool vec = p.hidden % 8 == 0;
  const int64_t items = p.tokens * (vec ? p.hidden / 8 : p.hidden);
  const int64_t want = (items + 255) / 256, most = static_cast<int64_t>(sms) * 16;
  const dim3 grid(static_cast<unsigned>(want < most ? want : most));
  auto go = [&](auto kernel) { return launch(kernel, grid, 256, 0, stream, pdl, p); };
  if (p.weight) {
    if (bf16)
      return vec ? go(moe_gather_kernel<__nv_bfloat16, 8, true>)
                 : go(moe_gather_kernel<__nv_bfloat16, 1, true>);
    return vec ? go(moe_gather_kernel<__half, 8, true>) : go(moe_gather_kernel<__half, 1, true>);
  }
  if (bf16)
    return vec ? go(moe_gather_kernel<__nv_bfloat16, 8, false>)
               : go(moe_gather_kernel<__nv_bfloat16, 1, false>);
  return vec ? go(moe_gather_kernel<__half, 8, false>) : go(moe_gather_kernel<__half, 1, false>);
}

cudaError_t launch_moe_combine_grad(const GatherParams& p, int bf16, cudaStream_t stream,
                                    int pdl) {
  const dim3 grid(static_cast<unsigned>(p.tokens));
  const bool vec = p.hidden % 8 == 0;
  auto go = [&](auto kernel) { return launch(kernel, grid, kGradThreads, 0, stream, pdl, p); };
  if (bf16)
    return vec ? go(moe_combine_grad_kernel<__nv_bfloat16, 8>)
               : go(moe_combine_grad_kernel<__nv_bfloat16, 1>);
  return vec ? go(moe_combine_grad_kernel<__half, 8>) : go(moe_combine_grad_kernel<__half, 1>);
}

cudaError_t launch_fp8_quantize(int64_t m, int64_t k, int bf16, int block_rows, const void* x,
                                void* q, float* scale, int sms, cudaStream_t stream, int pdl) {
  const uint4* src = static_cast<const uint4*>(x);
  uint4* dst = static_cast<uint4*>(q);
  const int64_t blocks_k = (k + 127) / 128;
  if (block_rows == 128) {
    const dim3 grid(static_cast<unsigned>((m + 127) / 128 * blocks_k));
    auto go = [&](auto kernel) {
      return launch(kernel, grid, 256, 0, stream, pdl, m, k, static_cast<int>(blocks_k), src, dst,
                    scale);
    };
    return bf16 ? go(quantize_blocks_kernel<__nv_bfloat16>) : go(quantize_blocks_kernel<__half>);
  }
  const int64_t want = (m * blocks_k * 8 + 255) / 256, most = static_cast<int64_t>(sms) * 16;
  const dim3 grid(static_cast<unsigned>(want < most ? want : most));
  auto go = [&](auto kernel) {
    return launch(kernel, grid, 256, 0, stream, pdl, m, k, src, dst, scale);
  };
  return bf16 ? go(quantize_rows_kernel<__nv_bfloat16>) : go(quantize_rows_kernel<__half>);
}

}  // namespace gf
