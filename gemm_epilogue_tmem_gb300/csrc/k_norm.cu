// Root-mean-square norm with the residual's addition before it: few rows, and rows
// that are not whole 16-byte words.
//
// A CTA loads its rows itself and keeps them in registers, in 16 bits, between their sum
// and the output. 16-byte accesses for rows of any length: where rows do not start on
// 16 bytes, the row's words are those it would have in an aligned array, the ones at its
// two ends are read and written one element at a time. HBM bounds both directions (one
// row: latency); nothing is kept from the forward but r itself, whose sum of squares the
// backward forms along with the other one that it needs. A row of 5120 takes 2.6 us, 5003
// rows of 2047 19.3 us (4.3 TB/s).
#include "norm_common.cuh"

namespace gf {
namespace {

// A row of a dense [rows, n] matrix of 16-bit elements as 16-byte words. ALIGNED:
// n is a multiple of 8; else the row begins at element `o` of its first word.
template <typename T, bool ALIGNED>
struct Row {
  int64_t word0;  // index of the first word
  int o, n, words;
  __device__ __forceinline__ Row(int64_t row, int n_) : n(n_) {
    const int64_t first = row * n_;
    o = ALIGNED ? 0 : static_cast<int>(first & 7);
    word0 = (first - o) >> 3;
    words = (o + n + 7) >> 3;
  }
  __device__ __forceinline__ bool whole(int w) const {
    return ALIGNED || ((w > 0 || o == 0) && 8 * w + 8 <= o + n);
  }
  __device__ __forceinline__ uint4 load(const void* base, int w) const {
    const uint4* at = static_cast<const uint4*>(base) + word0 + w;
    if (whole(w)) return *at;
    uint32_t v[4] = {0u, 0u, 0u, 0u};
    const uint16_t* e = reinterpret_cast<const uint16_t*>(at);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = 8 * w + j - o;
      if (col >= 0 && col < n) v[j / 2] |= static_cast<uint32_t>(e[j]) << (16 * (j & 1));
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
  }
  __device__ __forceinline__ void store(void* base, int w, const uint4& u) const {
    uint4* at = static_cast<uint4*>(base) + word0 + w;
    if (whole(w)) {
      *at = u;
      return;
    }
    const uint32_t v[4] = {u.x, u.y, u.z, u.w};
    uint16_t* e = reinterpret_cast<uint16_t*>(at);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = 8 * w + j - o;
      if (col >= 0 && col < n) e[j] = static_cast<uint16_t>(v[j / 2] >> (16 * (j & 1)));
    }
  }
  // a vector over the columns (the norm's weight), at this row's words
  __device__ __forceinline__ uint4 load_cols(const void* base, int w) const {
    if (ALIGNED) return static_cast<const uint4*>(base)[w];
    uint32_t v[4] = {0u, 0u, 0u, 0u};
    const uint16_t* e = static_cast<const uint16_t*>(base);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = 8 * w + j - o;
      if (col >= 0 && col < n) v[j / 2] |= static_cast<uint32_t>(e[col]) << (16 * (j & 1));
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
  }
};

// the sum over the blockDim.x threads of a row, in the same order in each of them
template <typename S>
__device__ __forceinline__ S row_sum(S s, S* red) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) s.add(s.other(d));
  const int warps = blockDim.x >> 5;
  if (warps == 1) return s;
  S* mine = red + threadIdx.y * warps;
  if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = s;
  __syncthreads();
  s = mine[0];
  for (int i = 1; i < warps; ++i) s.add(mine[i]);
  return s;
}

// Threads (x: the words of a row, y: rows). V words a thread.
template <typename T, int V, bool ALIGNED, bool FP8>
__global__ void __launch_bounds__(544) norm_kernel(const NormParams p) {
  __shared__ Sum<FP8> red[32];
  grid_dep_wait();
  grid_dep_launch();
  const int64_t at = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const Row<T, ALIGNED> row(at, p.hidden);
  const int words = at < p.rows ? row.words : 0;
  const int step = blockDim.x, w0 = threadIdx.x;
  uint4 r[V], wt[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int w = w0 + i * step;
    r[i] = w < words ? row.load(p.x, w) : make_uint4(0u, 0u, 0u, 0u);
  }
  if (p.residual != nullptr) {
    uint4 add[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int w = w0 + i * step;
      add[i] = w < words ? row.load(p.residual, w) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      r[i] = add8<T>(r[i], add[i]);  // the stream is kept in 16 bits, and normed as it is kept
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int w = w0 + i * step;
    wt[i] = w < words ? row.load_cols(p.weight, w) : make_uint4(0u, 0u, 0u, 0u);
  }
  if (p.residual_out != nullptr) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int w = w0 + i * step;
      if (w < words) row.store(p.residual_out, w, r[i]);
    }
  }
  Sum<FP8> s = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float f[8];
    unpack<T>(r[i], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) s.add(__fmul_rn(f[j], f[j]));
  }
  s = row_sum(s, red);
  float lo;
  const float rstd = inv_rms<FP8>(s, p.hidden, p.eps, lo);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int w = w0 + i * step;
    float f[8], g[8];
    unpack<T>(r[i], f);
    unpack<T>(wt[i], g);
    uint32_t mag = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f[j] *= g[j];
      if (FP8) mag = max(mag, finite_mag_bits(f[j]));
      f[j] *= rstd;
    }
    if ((!FP8 || p.out != nullptr) && w < words) row.store(p.out, w, pack<T>(f));
    if constexpr (FP8) {
      // 16 lanes hold a block of 128
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, d));
      float inv;
      const float scale = e4m3_scale(exact_mag(__uint_as_float(mag), rstd, lo), inv);
      if (w < words) {
        reinterpret_cast<uint2*>(p.out8)[row.word0 + w] =
            make_uint2(e4m3x4(f[0], f[1], f[2], f[3], inv), e4m3x4(f[4], f[5], f[6], f[7], inv));
        if ((threadIdx.x & 15) == 0) p.scale[at * ((p.hidden + 127) >> 7) + (w >> 4)] = scale;
      }
    }
  }
}

// ----------------------------------------------------------------- backward
// CTAs walk over the rows, a thread keeping the same columns from row to row for
// the weight's gradient (in registers; from V = 8 on in shared memory). Rows whose
// words do not begin on the row begin elsewhere in their first word each time,
// with a period of 8: there the thread rows of the grid are a multiple of 8.
template <typename T, int V, bool ALIGNED>
__global__ void __launch_bounds__(544) norm_grad_kernel(const NormParams p) {
  constexpr bool kSmemAcc = V >= 8;
  extern __shared__ float cols[];  // [hidden]
  __shared__ Sum2 red[2][32];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = blockIdx.x * blockDim.y + threadIdx.y;  // thread row
  const int step = blockDim.x, w0 = threadIdx.x;
  const bool sums = p.partials != nullptr;
  if (sums) {
    for (int c = threadIdx.y * blockDim.x + threadIdx.x; c < p.hidden; c += blockDim.x * blockDim.y)
      cols[c] = 0.f;
  }
  __syncthreads();
  float acc[kSmemAcc ? 1 : V][8];
#pragma unroll
  for (int i = 0; i < (kSmemAcc ? 1 : V); ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  const int o0 = ALIGNED ? 0 : static_cast<int>((static_cast<int64_t>(lane) * p.hidden) & 7);
  int turn = 0;
  // every thread row of a CTA goes through as many rows (barriers), the last past the end
  const int64_t cta_first = static_cast<int64_t>(blockIdx.x) * blockDim.y;
  for (int64_t skip = 0; cta_first + skip < p.rows; skip += p.lanes, turn ^= 1) {
    const int64_t at = lane + skip;
    const Row<T, ALIGNED> row(at, p.hidden);
    const int words = at < p.rows ? row.words : 0;
    uint4 r[V], dy[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int w = w0 + i * step;
      r[i] = dy[i] = make_uint4(0u, 0u, 0u, 0u);
      if (w < words) {
        r[i] = row.load(p.x, w);
        dy[i] = row.load(p.d_out, w);
      }
    }
    Sum2 s = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int w = w0 + i * step;
      float f[8], g[8], wt[8];
      unpack<T>(r[i], f);
      unpack<T>(dy[i], g);
      unpack<T>(w < words ? row.load_cols(p.weight, w) : make_uint4(0u, 0u, 0u, 0u), wt);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s.rr += f[j] * f[j];
        s.gr += g[j] * wt[j] * f[j];
      }
    }
    s = row_sum(s, red[turn]);
    const float n = static_cast<float>(p.hidden);
    const float rstd = rsqrtf(s.rr / n + p.eps);
    const float c = rstd * rstd * (s.gr / n);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int w = w0 + i * step;
      if (w < words) {
        float f[8], g[8], wt[8], d[8];
        unpack<T>(r[i], f);
        unpack<T>(dy[i], g);
        unpack<T>(row.load_cols(p.weight, w), wt);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = rstd * (g[j] * wt[j] - f[j] * c);
        if (p.residual != nullptr) {
          float e[8];
          unpack<T>(row.load(p.residual, w), e);
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] += e[j];
        }
        row.store(p.out, w, pack<T>(d));
        if (sums) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float v = g[j] * f[j] * rstd;
            if constexpr (kSmemAcc) {
              const int col = 8 * w + j - row.o;
              if (ALIGNED || (col >= 0 && col < p.hidden)) cols[col] += v;
            } else {
              acc[i][j] += v;
            }
          }
        }
      }
    }
  }
  if (!sums) return;
  if constexpr (!kSmemAcc) {
    // the thread rows one after the other: a fixed order
    for (int y = 0; y < blockDim.y; ++y) {
      __syncthreads();
      if (threadIdx.y == y) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int col = 8 * (w0 + i * step) + j - o0;
            if (col >= 0 && col < p.hidden) cols[col] += acc[i][j];
          }
      }
    }
  }
  __syncthreads();
  float* out = p.partials + static_cast<int64_t>(blockIdx.x) * p.hidden;
  for (int c = threadIdx.y * blockDim.x + threadIdx.x; c < p.hidden; c += blockDim.x * blockDim.y)
    out[c] = cols[c];
}

// 32 columns a CTA, its warps the rows in turn
constexpr int kSlices = 32;
__global__ void __launch_bounds__(32 * kSlices) column_sums_kernel(const float* partials, int rows, int n,
                                                          float* out) {
  __shared__ float red[kSlices][33];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (col < n) {
#pragma unroll 8
    for (int r = slice; r < rows; r += kSlices) s += partials[static_cast<int64_t>(r) * n + col];
  }
  red[slice][lane] = s;
  __syncthreads();
  if (slice == 0 && col < n) {
#pragma unroll
    for (int k = 1; k < kSlices; ++k) s += red[k][lane];
    out[col] = s;
  }
}

// Words of a row (with one to spare where it may begin anywhere), words a thread,
// threads a row and rows a CTA. One word a thread for longer rows where they begin
// anywhere, as a word takes more instructions and registers there (5003 rows, one word
// against two, forward / backward: of 2047 19.3 / 36.6 against 20.7 / 45.2 us, of 3001
// 27.3 / 49.9 against 27.1 / 57.7, of 4099 38.2 / 72.8 against 37.3 / 80.7, but 300 rows
// of 4099 4.0 against 3.3; whole words, 300 rows of 4096: 2.5 against 2.3).
struct Shape {
  int v, threads, rows;
};

Shape norm_shape(int64_t hidden) {
  const int words = static_cast<int>((hidden + 7) / 8) + (hidden % 8 != 0 ? 1 : 0);
  Shape s;
  s.v = words <= (hidden % 8 != 0 ? 384 : 256) ? 1 : words <= 1024 ? 2 : words <= 2048 ? 4 : 8;
  s.threads = (words + s.v * 32 - 1) / (s.v * 32) * 32;
  s.rows = s.threads >= 128 ? 1 : 128 / s.threads;
  return s;
}

template <typename T, bool ALIGNED, bool FP8>
cudaError_t forward(const NormParams& p, cudaStream_t stream, int pdl) {
  const Shape s = norm_shape(p.hidden);
  const int64_t ctas = (static_cast<int64_t>(p.rows) + s.rows - 1) / s.rows;
  const dim3 grid(static_cast<unsigned>(ctas)), block(s.threads, s.rows);
  switch (s.v) {
    case 1: return launch_pdl(norm_kernel<T, 1, ALIGNED, FP8>, grid, block, 0, stream, pdl, p);
    case 2: return launch_pdl(norm_kernel<T, 2, ALIGNED, FP8>, grid, block, 0, stream, pdl, p);
    case 4: return launch_pdl(norm_kernel<T, 4, ALIGNED, FP8>, grid, block, 0, stream, pdl, p);
    case 8: return launch_pdl(norm_kernel<T, 8, ALIGNED, FP8>, grid, block, 0, stream, pdl, p);
  }
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t forward_type(const NormParams& p, cudaStream_t stream, int pdl) {
  if (p.out8 != nullptr) return forward<T, true, true>(p, stream, pdl);
  return p.hidden % 8 == 0 ? forward<T, true, false>(p, stream, pdl)
                           : forward<T, false, false>(p, stream, pdl);
}

// calls f(kernel) with the backward kernel of these rows
template <typename T, typename F>
cudaError_t with_grad_kernel(int64_t hidden, const F& f) {
  const bool aligned = hidden % 8 == 0;
  switch (norm_shape(hidden).v) {
    case 1: return f(aligned ? norm_grad_kernel<T, 1, true> : norm_grad_kernel<T, 1, false>);
    case 2: return f(aligned ? norm_grad_kernel<T, 2, true> : norm_grad_kernel<T, 2, false>);
    case 4: return f(aligned ? norm_grad_kernel<T, 4, true> : norm_grad_kernel<T, 4, false>);
    case 8: return f(aligned ? norm_grad_kernel<T, 8, true> : norm_grad_kernel<T, 8, false>);
  }
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t grad_ctas(int64_t rows, int64_t hidden, int sms, int* ctas) {
  const Shape s = norm_shape(hidden);
  return with_grad_kernel<T>(hidden, [&](auto kernel) {
    const size_t smem = static_cast<size_t>(hidden) * 4;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kNormMaxHidden * 4);
    if (e != cudaSuccess) return e;
    int per_sm = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, s.threads * s.rows, smem);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    int64_t n = (rows + s.rows - 1) / s.rows;
    const int64_t resident = static_cast<int64_t>(per_sm) * sms;
    const int64_t least = (n + kMostTurns - 1) / kMostTurns;
    if (n > resident) n = resident > least ? resident : least;
    if (hidden % 8 != 0) n = (n + 7) / 8 * 8;  // thread rows in whole periods
    *ctas = static_cast<int>(n < 1 ? 1 : n);
    return cudaSuccess;
  });
}

template <typename T>
cudaError_t backward(const NormParams& p, int ctas, cudaStream_t stream, int pdl) {
  const Shape s = norm_shape(p.hidden);
  NormParams q = p;
  q.lanes = ctas * s.rows;
  return with_grad_kernel<T>(p.hidden, [&](auto kernel) {
    return launch_pdl(kernel, dim3(ctas), dim3(s.threads, s.rows),
                      static_cast<size_t>(p.hidden) * 4, stream, pdl, q);
  });
}

}  // namespace

static bool streams(const NormParams& p, NormStream* s) {
  return norm_stream_shape(p.rows, p.hidden, p.residual != nullptr ? 2 : 1, p.out8 != nullptr, p.sms, s);
}

int64_t norm_ctas(const NormParams& p, int* rows, int* stages) {
  NormStream s;
  if (streams(p, &s)) {
    *rows = s.rows;
    *stages = s.stages;
    return s.ctas;
  }
  *rows = norm_shape(p.hidden).rows;
  *stages = 0;
  return (static_cast<int64_t>(p.rows) + *rows - 1) / *rows;
}

cudaError_t launch_norm(const NormParams& p, int bf16, cudaStream_t stream, int pdl) {
  NormStream s;
  if (streams(p, &s)) return launch_norm_stream(p, s, bf16, stream, pdl);
  return bf16 ? forward_type<__nv_bfloat16>(p, stream, pdl) : forward_type<__half>(p, stream, pdl);
}

int norm_grad_ctas(int64_t rows, int64_t hidden, int bf16, int sms, cudaError_t* err) {
  int n = 0;
  *err = bf16 ? grad_ctas<__nv_bfloat16>(rows, hidden, sms, &n)
              : grad_ctas<__half>(rows, hidden, sms, &n);
  return n;
}

int norm_grad_partials(int64_t rows, int64_t hidden, int sms, int ctas) {
  int most = ctas;
  NormStream s;
  for (int arrays = 2; arrays <= 3; ++arrays)
    if (norm_stream_shape(rows, hidden, arrays, false, sms, &s) && s.ctas > most) most = s.ctas;
  return most;
}

cudaError_t launch_norm_grad(const NormParams& p, int bf16, int ctas, cudaStream_t stream, int pdl,
                             int* partial_rows) {
  NormStream s;
  if (norm_stream_shape(p.rows, p.hidden, p.residual != nullptr ? 3 : 2, false, p.sms, &s)) {
    *partial_rows = s.ctas;
    return launch_norm_grad_stream(p, s, bf16, stream, pdl);
  }
  *partial_rows = ctas;
  return bf16 ? backward<__nv_bfloat16>(p, ctas, stream, pdl) : backward<__half>(p, ctas, stream, pdl);
}

cudaError_t launch_column_sums(const float* partials, int rows, int cols, float* out,
                               cudaStream_t stream, int pdl) {
  return launch_pdl(column_sums_kernel, dim3((static_cast<unsigned>(cols) + 31) / 32), dim3(32 * kSlices), 0, stream, pdl,
                    partials, rows, cols, out);
}

}  // namespace gf
