// d_z = d_out act'(z) and the gradient of the bias, the column sums of the fp32 d_z:
// the backward pass of out = act(A B + bias) + residual up to its product (the
// residual's gradient is d_out itself).
//
// One pass over d_out and z, bound by HBM (GELU of 8192 x 16384 123 us, 6.5 TB/s). A warp has 256 columns, 16 bytes a lane,
// and every eighth row of its CTA's chunk; a thread's columns stay
// the same, so their sums are in registers until the CTA's eight warps meet. The
// chunks' sums are added by a second kernel, in a fixed order.
#include "block.h"
#include "gemm_kernel.cuh"
#include "ptx.cuh"

namespace gf {
namespace {

constexpr int kPerSm = 4;  // CTAs of an SM
// rows of a chunk at most, an eighth of which fp32 adds up in a row: beside the sum of 2^18 of its
// size a term has 6 bits left
constexpr int64_t kMostRows = 65536;

// act'(z) of SiLU and GELU: with s = 1 / (1 + e^-u) and act = z s, s + z u' s (1 - s); u = z (SiLU) or
// 2 c (z + k z^3) (GELU's tanh form). e^-u by the hardware's exponential of base 2, the
// base in the constants, and its reciprocal, small results flushed. Where s has reached
// its end the second term is 0, also for an infinite z.
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  constexpr float kLog2e = 1.4426950408889634f;
  const float z2 = z * z;
  const float t = ACT == kActGelu ? z * fmaf(-2.f * kGeluCK * kLog2e, z2, -2.f * kGeluC * kLog2e)
                                  : z * -kLog2e;
  const float zdu = ACT == kActGelu ? z * fmaf(2.f * kGelu3CK, z2, 2.f * kGeluC) : z;
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
  const float w = fmaf(-s, s, s);
  return w == 0.f ? s : fmaf(zdu, w, s);
}

template <typename T, int ACT>
__global__ void __launch_bounds__(256, kPerSm) dact_kernel(const DactParams p) {
  // rows of a thread whose loads are in flight (GELU of 8192 x 16384 with two 123 us, with
  // four 128; sums alone 57 and 44)
  constexpr int kRowsInFlight = ACT == kActNone ? 4 : 2;
  __shared__ float red[8][256];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 256 + lane * 8;
  const int64_t end64 = static_cast<int64_t>(blockIdx.y + 1) * p.chunk_rows;
  const int end = end64 < p.rows ? static_cast<int>(end64) : p.rows;
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.f;
  if (col < p.cols) {
    for (int64_t row0 = static_cast<int64_t>(blockIdx.y) * p.chunk_rows + warp; row0 < end;
         row0 += 8 * kRowsInFlight) {
      uint4 dy[kRowsInFlight], z[kRowsInFlight];
#pragma unroll
      for (int i = 0; i < kRowsInFlight; ++i) {
        const int64_t at = ((row0 + 8 * i) * p.cols + col) >> 3;
        if (row0 + 8 * i < end) {
          dy[i] = static_cast<const uint4*>(p.d_out)[at];
          if (ACT != kActNone) z[i] = static_cast<const uint4*>(p.z)[at];
        }
      }
#pragma unroll
      for (int i = 0; i < kRowsInFlight; ++i) {
        if (row0 + 8 * i < end) {
          float d[8], f[8];
          unpack8<T>(dy[i], d);
          if constexpr (ACT != kActNone) {
            unpack8<T>(z[i], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if constexpr (ACT == kActRelu)
                d[j] = f[j] > 0.f ? d[j] : 0.f;  // (an infinite gradient too)
              else
                d[j] *= act_slope<ACT>(f[j]);
            }
            static_cast<uint4*>(p.d_z)[((row0 + 8 * i) * p.cols + col) >> 3] =
                make_uint4(pack2<T>(d[0], d[1]), pack2<T>(d[2], d[3]), pack2<T>(d[4], d[5]),
                           pack2<T>(d[6], d[7]));
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] += d[j];
        }
      }
    }
  }
  if (p.partials == nullptr) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) red[warp][lane * 8 + j] = acc[j];
  __syncthreads();
  const int mine = blockIdx.x * 256 + threadIdx.x;
  if (mine < p.cols) {
    float s = red[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < 8; ++w) s += red[w][threadIdx.x];
    p.partials[static_cast<int64_t>(blockIdx.y) * p.cols + mine] = s;
  }
}

template <typename T>
cudaError_t dact(const DactParams& p, int chunks, cudaStream_t stream, int pdl) {
  const dim3 grid((static_cast<unsigned>(p.cols) + 255) / 256, chunks), block(256);
  switch (p.act) {
    case kActNone: return launch_pdl(dact_kernel<T, kActNone>, grid, block, 0, stream, pdl, p);
    case kActRelu: return launch_pdl(dact_kernel<T, kActRelu>, grid, block, 0, stream, pdl, p);
    case kActGelu: return launch_pdl(dact_kernel<T, kActGelu>, grid, block, 0, stream, pdl, p);
    case kActSilu: return launch_pdl(dact_kernel<T, kActSilu>, grid, block, 0, stream, pdl, p);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

int dact_chunks(int64_t rows, int64_t cols, int sms) {
  const int64_t blocks = (cols + 255) / 256;
  int64_t chunks = static_cast<int64_t>(sms) * kPerSm / blocks;  // one wave of CTAs
  const int64_t least = (rows + kMostRows - 1) / kMostRows, most = (rows + 31) / 32;
  if (chunks < least) chunks = least;
  if (chunks > most) chunks = most;
  return static_cast<int>(chunks < 1 ? 1 : chunks);
}

cudaError_t launch_dact(const DactParams& p, int bf16, int chunks, cudaStream_t stream, int pdl) {
  return bf16 ? dact<__nv_bfloat16>(p, chunks, stream, pdl) : dact<__half>(p, chunks, stream, pdl);
}

}  // namespace gf
