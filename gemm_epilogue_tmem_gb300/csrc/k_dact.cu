// d_z = d_out act'(z) and the gradient of the bias, the column sums of the fp32 d_z:
// the backward pass of out = act(A B + bias) + residual up to its product (the
// residual's gradient is d_out itself).
//
// One pass over d_out and z, bound by HBM. A warp has 256 columns, 16 bytes a lane,
// and every eighth row of its CTA's chunk, four in flight; a thread's columns stay
// the same, so their sums are in registers until the CTA's eight warps meet. The
// chunks' sums are added by a second kernel, in a fixed order.
#include "block.h"
#include "gemm_kernel.cuh"
#include "ptx.cuh"

namespace gf {
namespace {

constexpr int kRowsInFlight = 4;

// act'(z), with s = 1 / (1 + e^-u) and act = z s: s + z s (1 - s) u'
__device__ __forceinline__ float act_slope(int act, float z) {
  if (act == kActRelu) return z > 0.f ? 1.f : 0.f;
  float u = z, du = 1.f;
  if (act == kActGelu) {
    u = z * fmaf(2.f * kGeluCK, z * z, 2.f * kGeluC);
    du = fmaf(2.f * kGelu3CK, z * z, 2.f * kGeluC);
  }
  const float s = logistic_f(u);
  // where the logistic has reached its end the second term is 0, also for an infinite z
  const float t = s * (1.f - s);
  return t == 0.f ? s : fmaf(z * du, t, s);
}

template <typename T, int ACT>
__global__ void __launch_bounds__(256) dact_kernel(const DactParams p) {
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
            for (int j = 0; j < 8; ++j) d[j] *= act_slope(ACT, f[j]);
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
  const dim3 grid((p.cols + 255) / 256, chunks), block(256);
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
  int64_t chunks = static_cast<int64_t>(sms) * 4 / blocks;  // one wave of CTAs
  const int64_t most = (rows + 8 * kRowsInFlight - 1) / (8 * kRowsInFlight);
  if (chunks > most) chunks = most;
  return static_cast<int>(chunks < 1 ? 1 : chunks);
}

cudaError_t launch_dact(const DactParams& p, int bf16, int chunks, cudaStream_t stream, int pdl) {
  return bf16 ? dact<__nv_bfloat16>(p, chunks, stream, pdl) : dact<__half>(p, chunks, stream, pdl);
}

}  // namespace gf
