// The root-mean-square norm of many rows of whole 16-byte words.
//
// CTAs that stay walk over the rows, which bulk copies bring to a ring in shared memory
// several rows ahead, so that HBM, which bounds both directions, is asked for the next
// rows while the sum of one is formed. Groups of blockDim.y consecutive rows (short ones
// share a CTA) are the turns of CTA blockIdx.x, blockIdx.x + gridDim.x, ...; a stage of
// the ring holds a group of two or three arrays, each brought by one copy. A turn has one
// barrier, that of the row's sum: after it every thread has done with the stage of
// the turn before, which is filled again.
//
// A thread has the same columns in every turn: the weight stays in its registers, and
// so do the column sums of the weight's gradient. 16384 x 5120 with a residual to e4m3
// 92 us (6.4 TB/s), the gradient of 16384 x 4096 88 us (6.1 TB/s); to e4m3 without a
// residual, half the bytes, instructions bound it (some 26 an element, 76 us).
#include "norm_common.cuh"

namespace gf {
namespace {

constexpr int kMaxStages = 8;
// Turns of a CTA from which on rows stream (us, without the ring and with it, rows from HBM, to
// e4m3: 1140 x 2048 5.4 and 4.7, 684 x 4096 6.0 and 5.1, 1216 x 8192 17.4 and 12.1. In 16 bits it
// pays later: 1216 x 8192 11.3 and 10.9, 3648 x 5120 18.5 and 18.1, but 3648 x 4096 14.4 and 15.5, 6080 x
// 2048 12.0 and 15.7; gradient 912 x 8192 14.7 and 14.1, 3648 x 5120 27.1 and 25.8, 3648 x 4096 20.1 and
// 21.5).
constexpr int kLeastTurns = 2;
constexpr size_t kStreamSmem = 216 * 1024;  // of an SM, for rings
// by the words of a thread: most threads of a CTA, CTAs of an SM
constexpr int stream_threads(int v) { return v == 1 ? 256 : 512; }
constexpr int stream_per_sm(int v) { return v == 1 ? 5 : v == 2 ? 2 : 1; }

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

struct Ring {
  uint32_t data, full;   // shared-memory addresses: the stages, their barriers
  volatile int* stop;
  uint32_t array_bytes;  // of one array of a stage
  int arrays, stages;
  int64_t groups;

  __device__ __forceinline__ void start(const NormParams& p, int arrays_, uint8_t* smem, uint64_t* bars,
                                        int* flag) {
    data = smem_u32(smem);
    full = smem_u32(bars);
    stop = flag;
    arrays = arrays_;
    stages = p.stages;
    array_bytes = blockDim.y * static_cast<uint32_t>(p.hidden) * 2u;
    groups = (static_cast<int64_t>(p.rows) + blockDim.y - 1) / blockDim.y;
    if (leader()) {
      for (int s = 0; s < stages; ++s) mbar_init(full + 8u * s, 1);
      *flag = 0;
      fence_mbar_init();
    }
    __syncthreads();
    grid_dep_wait();
    grid_dep_launch();
    if (leader())
      for (int s = 0; s < stages; ++s)
        issue(p, s, blockIdx.x + static_cast<int64_t>(s) * gridDim.x);
  }
  __device__ __forceinline__ bool leader() const { return threadIdx.x == 0 && threadIdx.y == 0; }
  __device__ __forceinline__ uint32_t array(int stage, int a) const {
    return data + static_cast<uint32_t>(stage * arrays + a) * array_bytes;
  }
  // a group's rows of each array into the stage; nothing past the last group
  __device__ __forceinline__ void issue(const NormParams& p, int stage, int64_t group) const {
    if (group >= groups) return;
    if (p.drop_load != 0 && (group - blockIdx.x) / gridDim.x + 1 == p.drop_load) return;
    const int64_t row = group * blockDim.y, left = p.rows - row;
    const int rows = left < blockDim.y ? static_cast<int>(left) : static_cast<int>(blockDim.y);
    const uint32_t bytes = static_cast<uint32_t>(rows) * static_cast<uint32_t>(p.hidden) * 2u;
    const uint32_t bar = full + 8u * static_cast<uint32_t>(stage);
    const int64_t at = row * p.hidden * 2;
    mbar_arrive_expect_tx(bar, bytes * static_cast<uint32_t>(arrays));
    bulk_load(array(stage, 0), static_cast<const char*>(p.x) + at, bytes, bar);
    if (p.d_out != nullptr)
      bulk_load(array(stage, 1), static_cast<const char*>(p.d_out) + at, bytes, bar);
    if (p.residual != nullptr)
      bulk_load(array(stage, arrays - 1), static_cast<const char*>(p.residual) + at, bytes, bar);
  }
  __device__ __forceinline__ void wait(const NormParams& p, int stage, uint32_t phase) const {
    if (!mbar_wait_bounded(full + 8u * static_cast<uint32_t>(stage), phase, stop, p.wait_limit_ns)) {
      *stop = 1;  // the waits that follow end at once; outputs are incomplete
      atomicOr(p.status, 1);
    }
  }
  // a CTA that gave up may still have copies in flight towards its shared memory
  __device__ __forceinline__ void finish() const {
    if (__syncthreads_or(*stop)) sleep_ns(200000);
  }
};

// the sum over a row's threads, with the turn's one barrier
template <typename S>
__device__ __forceinline__ S turn_sum(S s, S* red) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) s.add(s.other(d));
  const int warps = blockDim.x >> 5;
  S* mine = red + threadIdx.y * warps;
  if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = s;
  __syncthreads();
  s = mine[0];
#pragma unroll 4
  for (int i = 1; i < warps; ++i) s.add(mine[i]);
  return s;
}

// exact_mag with the row's sum formed anew, in two fp32, by one warp from the ring
template <typename T>
__device__ __noinline__ uint32_t sure_mag(const NormParams& p, uint32_t x, uint32_t residual, float mag) {
  Sum<true> s = {0.f, 0.f};
  for (int w = threadIdx.x & 31; w < p.hidden / 8; w += 32) {
    uint4 v = ld_shared_v4(x + 16u * static_cast<uint32_t>(w));
    if (residual != 0u) v = add8<T>(v, ld_shared_v4(residual + 16u * static_cast<uint32_t>(w)));
    float f[8];
    unpack<T>(v, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) s.add(__fmul_rn(f[j], f[j]));
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) s.add(s.other(d));
  float lo;
  const float hi = inv_rms<true>(s, p.hidden, p.eps, lo);
  return exact_mag(mag, hi, lo);
}

// e4m3: a thread has pairs of words, 16 columns, so that 8 lanes hold a block of 128.
template <typename T, int V, bool FP8>
__global__ void __launch_bounds__(stream_threads(V), stream_per_sm(V))
    norm_stream_kernel(const __grid_constant__ NormParams p) {
  static_assert(!FP8 || V % 2 == 0, "pairs of words");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Sum<false> red[2][32];
  __shared__ uint64_t full[kMaxStages];
  __shared__ int stop;
  const int words = p.hidden >> 3, step = blockDim.x;
  auto word = [&](int i) {
    return FP8 ? 2 * (static_cast<int>(threadIdx.x) + (i >> 1) * step) + (i & 1)
               : static_cast<int>(threadIdx.x) + i * step;
  };
  Ring ring;
  ring.start(p, p.residual != nullptr ? 2 : 1, smem, full, &stop);
  uint4 wt[V];
#pragma unroll
  for (int i = 0; i < V; ++i)
    wt[i] = word(i) < words ? static_cast<const uint4*>(p.weight)[word(i)] : make_uint4(0u, 0u, 0u, 0u);
  const float inv_n = 1.f / static_cast<float>(p.hidden);
  int stage = 0, turn = 0;
  uint32_t phase = 0;
  for (int64_t group = blockIdx.x; group < ring.groups; group += gridDim.x, turn ^= 1) {
    ring.wait(p, stage, phase);
    const int64_t at = group * blockDim.y + threadIdx.y;
    const bool row_ok = at < p.rows;
    const uint32_t row_off = threadIdx.y * static_cast<uint32_t>(p.hidden) * 2u;
    const uint32_t x = ring.array(stage, 0) + row_off;
    const uint32_t residual = p.residual != nullptr ? ring.array(stage, 1) + row_off : 0u;
    const int64_t word0 = at * words;
    uint4 r[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
      r[i] = row_ok && word(i) < words ? ld_shared_v4(x + 16u * static_cast<uint32_t>(word(i)))
                                       : make_uint4(0u, 0u, 0u, 0u);
    if (residual != 0u) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (row_ok && word(i) < words) {
          r[i] = add8<T>(r[i], ld_shared_v4(residual + 16u * static_cast<uint32_t>(word(i))));
          if (p.residual_out != nullptr) static_cast<uint4*>(p.residual_out)[word0 + word(i)] = r[i];
        }
      }
    }
    Sum<false> s = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float f[8];
      unpack<T>(r[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) s.hi = fmaf(f[j], f[j], s.hi);
    }
    s = turn_sum(s, red[turn]);
    if (ring.leader() && group != blockIdx.x)
      ring.issue(p, stage == 0 ? ring.stages - 1 : stage - 1,
                 group + static_cast<int64_t>(ring.stages - 1) * gridDim.x);
    const float var = fmaf(s.hi, inv_n, p.eps);
    float rstd = rsqrtf(var);
    if constexpr (FP8) {  // one step of Newton's method: an error moves values over e4m3's borders
      const float e = fmaf(-var * rstd, rstd, 1.f);
      if (fabsf(e) < 1e-3f) rstd = fmaf(0.5f * rstd, e, rstd);  // (not of 0 or infinity)
    }
    if constexpr (!FP8) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float f[8], g[8];
        unpack<T>(r[i], f);
        unpack<T>(wt[i], g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = f[j] * g[j] * rstd;
        if (row_ok && word(i) < words) static_cast<uint4*>(p.out)[word0 + word(i)] = pack<T>(f);
      }
    } else {
#pragma unroll
      for (int u = 0; u < V / 2; ++u) {
        const bool here = row_ok && word(2 * u) < words;
        float f[16];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float a[8], g[8];
          unpack<T>(r[2 * u + h], a);
          unpack<T>(wt[2 * u + h], g);
#pragma unroll
          for (int j = 0; j < 8; ++j) f[8 * h + j] = a[j] * g[j];
        }
        if (p.out != nullptr && here) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = f[8 * h + j] * rstd;
            static_cast<uint4*>(p.out)[word0 + word(2 * u + h)] = pack<T>(y);
          }
        }
        float mag = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) mag = fmaxf(mag, fabsf(f[j]));  // (NaN left out)
        uint32_t m = __float_as_uint(mag);
        const bool finite = __all_sync(0xFFFFFFFFu, m < 0x7F800000u && s.hi < INFINITY);
        if (!finite) {  // the finite ones' alone
          m = 0u;
#pragma unroll
          for (int j = 0; j < 16; ++j) m = max(m, finite_mag_bits(f[j]));
        }
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
        uint32_t bits = finite_mag_bits(__uint_as_float(m) * rstd);
        // Next to the border of two scales: rstd is of fp32 sums of 8 V + 22 additions, half
        // of whose error it has, a product and a root, 2^-18 at most; 64 is 2^-17.8.
        const bool doubt = row_ok && abs(static_cast<int>(bits & 0x7FFFFFu) - 0x600000) <= 64;
        if (__any_sync(0xFFFFFFFFu, doubt)) {
          const uint32_t sure = sure_mag<T>(p, x, residual, __uint_as_float(m));
          if (doubt) bits = sure;
        }
        float inv;
        const float scale = e4m3_scale(bits, inv);
        uint4 q;
        const float both = rstd * inv;  // (inv a power of two: rounded as f * rstd is)
        if (finite && both < INFINITY) {
          q = quant16<true>(f, both);
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) f[j] *= rstd;
          q = quant16<false>(f, inv);
        }
        if (here) {
          reinterpret_cast<uint4*>(p.out8)[(word0 + word(2 * u)) >> 1] = q;
          if ((threadIdx.x & 7) == 0)
            p.scale[at * ((p.hidden + 127) >> 7) + (word(2 * u) >> 4)] = scale;
        }
      }
    }
    if (++stage == ring.stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  ring.finish();
}

template <typename T, int V>
__global__ void __launch_bounds__(stream_threads(V), stream_per_sm(V))
    norm_grad_stream_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Sum2 red[2][32];
  __shared__ uint64_t full[kMaxStages];
  __shared__ int stop;
  const int words = p.hidden >> 3, step = blockDim.x, w0 = threadIdx.x;
  Ring ring;
  ring.start(p, p.residual != nullptr ? 3 : 2, smem, full, &stop);
  uint4 wt[V];
  const float inv_n = 1.f / static_cast<float>(p.hidden);
  float acc[V][8];  // the weight's gradient, of this thread's columns
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int w = w0 + i * step;
    wt[i] = w < words ? static_cast<const uint4*>(p.weight)[w] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  }
  int stage = 0, turn = 0;
  uint32_t phase = 0;
  for (int64_t group = blockIdx.x; group < ring.groups; group += gridDim.x, turn ^= 1) {
    ring.wait(p, stage, phase);
    const int64_t at = group * blockDim.y + threadIdx.y;
    const bool row_ok = at < p.rows;
    const uint32_t row_off = threadIdx.y * static_cast<uint32_t>(p.hidden) * 2u;
    const uint32_t x = ring.array(stage, 0) + row_off, dy = ring.array(stage, 1) + row_off;
    const uint32_t along = ring.array(stage, 2) + row_off;
    Sum2 s = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int w = w0 + i * step;
      if (row_ok && w < words) {
        float f[8], g[8], wf[8];
        unpack<T>(ld_shared_v4(x + 16u * static_cast<uint32_t>(w)), f);
        unpack<T>(ld_shared_v4(dy + 16u * static_cast<uint32_t>(w)), g);
        unpack<T>(wt[i], wf);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s.rr = fmaf(f[j], f[j], s.rr);
          s.gr = fmaf(g[j] * wf[j], f[j], s.gr);
        }
      }
    }
    s = turn_sum(s, red[turn]);
    if (ring.leader() && group != blockIdx.x)
      ring.issue(p, stage == 0 ? ring.stages - 1 : stage - 1,
                 group + static_cast<int64_t>(ring.stages - 1) * gridDim.x);
    const float rstd = rsqrtf(fmaf(s.rr, inv_n, p.eps));
    const float c = rstd * rstd * (s.gr * inv_n);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int w = w0 + i * step;
      if (row_ok && w < words) {
        float f[8], g[8], wf[8], d[8];
        unpack<T>(ld_shared_v4(x + 16u * static_cast<uint32_t>(w)), f);
        unpack<T>(ld_shared_v4(dy + 16u * static_cast<uint32_t>(w)), g);
        unpack<T>(wt[i], wf);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          d[j] = rstd * (g[j] * wf[j] - f[j] * c);
          acc[i][j] = fmaf(g[j] * f[j], rstd, acc[i][j]);
        }
        if (p.residual != nullptr) {
          float e[8];
          unpack<T>(ld_shared_v4(along + 16u * static_cast<uint32_t>(w)), e);
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] += e[j];
        }
        static_cast<uint4*>(p.out)[at * words + w] = pack<T>(d);
      }
    }
    if (++stage == ring.stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  ring.finish();
  if (p.partials == nullptr) return;
  // the thread rows one after the other, a fixed order, in the ring's memory
  float* cols = reinterpret_cast<float*>(smem);
  for (int y = 0; y < blockDim.y; ++y) {
    if (threadIdx.y == y) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int w = w0 + i * step;
        if (w < words) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            cols[8 * w + j] = acc[i][j] + (y > 0 ? cols[8 * w + j] : 0.f);
        }
      }
    }
    __syncthreads();
  }
  float* out = p.partials + static_cast<int64_t>(blockIdx.x) * p.hidden;
  for (int c = threadIdx.y * blockDim.x + threadIdx.x; c < p.hidden; c += blockDim.x * blockDim.y)
    out[c] = cols[c];
}

template <typename K>
cudaError_t launch_ring(K kernel, const NormParams& p, const NormStream& s, cudaStream_t stream, int pdl) {
  // (always the same amount: it belongs to the kernel, which another thread may be launching
  // with the ring of other rows)
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kStreamSmem));
  if (e != cudaSuccess) return e;
  NormParams q = p;
  q.stages = s.stages;
  return launch_pdl(kernel, dim3(s.ctas), dim3(s.threads, s.rows), s.smem, stream, pdl, q);
}

template <typename T, bool FP8>
cudaError_t forward(const NormParams& p, const NormStream& s, cudaStream_t stream, int pdl) {
  switch (s.v) {
    case 1:
      if constexpr (!FP8) return launch_ring(norm_stream_kernel<T, 1, FP8>, p, s, stream, pdl);
      break;
    case 2: return launch_ring(norm_stream_kernel<T, 2, FP8>, p, s, stream, pdl);
    case 4: return launch_ring(norm_stream_kernel<T, 4, FP8>, p, s, stream, pdl);
    case 8: return launch_ring(norm_stream_kernel<T, 8, FP8>, p, s, stream, pdl);
  }
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t backward(const NormParams& p, const NormStream& s, cudaStream_t stream, int pdl) {
  switch (s.v) {
    case 1: return launch_ring(norm_grad_stream_kernel<T, 1>, p, s, stream, pdl);
    case 2: return launch_ring(norm_grad_stream_kernel<T, 2>, p, s, stream, pdl);
    case 4: return launch_ring(norm_grad_stream_kernel<T, 4>, p, s, stream, pdl);
    case 8: return launch_ring(norm_grad_stream_kernel<T, 8>, p, s, stream, pdl);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

// About 256 threads a CTA, and as many CTAs an SM as there are registers for and rings of
// two stages fit: a turn is a chain of latencies that others fill. Not for rows that give a CTA no second
// turn, nor for those of which a ring does not hold two.
bool norm_stream_shape(int64_t rows, int64_t hidden, int arrays, bool pairs, int sms, NormStream* s) {
  if (hidden % 8 != 0) return false;
  const int words = static_cast<int>(hidden / 8);
  s->v = words <= 256 && !pairs ? 1 : words <= 1024 ? 2 : words <= 2048 ? 4 : 8;
  s->threads = (words + s->v * 32 - 1) / (s->v * 32) * 32;
  s->rows = s->threads >= 192 ? 1 : 256 / s->threads;
  const size_t stage = static_cast<size_t>(s->rows) * words * 16 * arrays;
  // (two CTAs an SM and three: 16384 x 5120 to e4m3 with a residual 94 and 104 us, without
  // one 77 and 75, 16384 x 4096 81 and 59; backward 90 and 85)
  int per_sm = s->v == 2 && s->threads <= 320 && (!pairs || arrays == 1) ? 3 : stream_per_sm(s->v);
  while (per_sm > 1 && per_sm * 2 * stage > kStreamSmem) --per_sm;
  s->stages = static_cast<int>(kStreamSmem / per_sm / stage);
  if (s->stages > kMaxStages) s->stages = kMaxStages;
  if (s->stages < 2) return false;
  s->smem = s->stages * stage;
  const int64_t groups = (rows + s->rows - 1) / s->rows, most = static_cast<int64_t>(per_sm) * sms;
  // as many turns for every CTA, but for one
  int64_t turns = (groups + most - 1) / most;
  if (turns > kMostTurns) turns = kMostTurns;
  s->ctas = static_cast<int>(turns > 0 ? (groups + turns - 1) / turns : 0);
  return turns >= kLeastTurns;
}

cudaError_t launch_norm_stream(const NormParams& p, const NormStream& s, int bf16, cudaStream_t stream,
                               int pdl) {
  if (p.out8 != nullptr)
    return bf16 ? forward<__nv_bfloat16, true>(p, s, stream, pdl) : forward<__half, true>(p, s, stream, pdl);
  return bf16 ? forward<__nv_bfloat16, false>(p, s, stream, pdl) : forward<__half, false>(p, s, stream, pdl);
}

cudaError_t launch_norm_grad_stream(const NormParams& p, const NormStream& s, int bf16,
                                    cudaStream_t stream, int pdl) {
  return bf16 ? backward<__nv_bfloat16>(p, s, stream, pdl) : backward<__half>(p, s, stream, pdl);
}

}  // namespace gf
