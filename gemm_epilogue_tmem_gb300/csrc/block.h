// Host-side view of the kernels around the products of a pre-norm block: the
// router's choice, the root-mean-square norm, the gradient of an activation and
// its bias.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gf {

// ------------------------------------------------------------------- router
struct RouteParams {
  int32_t tokens, experts, topk;
  int32_t groups, group_size, topk_groups;
  int32_t group_best;   // a group's score: its best, or the sum of its two best
  int32_t sigmoid;      // 0: softmax
  int32_t renorm;
  float scale;
  int64_t ld;           // elements between rows of logits and of d_logits
  // set by the launcher: a power of two of lanes, 1 << lane_shift, share a group; the
  // experts of each
  int32_t lane_shift, per_lane;
  int32_t sms;
  int32_t vector;       // 1: a lane's experts are loaded in words (aligned, none missing)
  const void* logits;
  const float* bias;    // NULL: none
  int32_t* expert;      // forward: out; backward: in
  float* weight;
  const float* d_weight;
  void* d_logits;
};

constexpr int kRouteMaxGroups = 32;

// logits: 0 fp16, 1 bf16, 2 fp32
cudaError_t launch_route(const RouteParams& p, int type, cudaStream_t stream, int pdl);
// the CTAs of that launch, and the tokens that each has at a time
int64_t route_ctas(const RouteParams& p, int type, int* tokens);
cudaError_t launch_route_grad(const RouteParams& p, int type, cudaStream_t stream, int pdl);

// --------------------------------------------------------------------- norm
constexpr int kNormMaxHidden = 32768;

struct NormParams {
  int32_t rows, hidden;
  float eps;
  int32_t lanes;        // backward: rows in work at a time, a column sum each
  int32_t sms;
  int32_t stages;       // of a streaming kernel's ring
  int32_t* status;
  uint64_t wait_limit_ns;
  int32_t drop_load;    // test hook: 1-based index of a CTA's stage load to skip (0: none)
  const void* x;        // backward: the rows that were normed
  const void* residual; // backward: the gradient that comes along the residual
  const void* weight;
  void* residual_out;
  void* out;            // backward: d_x
  uint8_t* out8;
  float* scale;
  const void* d_out;
  float* partials;      // backward: [partial rows][hidden]; NULL: no gradient of the weight
};

cudaError_t launch_norm(const NormParams& p, int bf16, cudaStream_t stream, int pdl);
// the CTAs of that launch, the rows that each has at a time, and its ring's stages (0: no ring)
int64_t norm_ctas(const NormParams& p, int* rows, int* stages);
// The CTAs of the backward kernel that loads its rows itself, for so many (0 with an
// error in *err), and the most rows of partial sums of either backward kernel.
int norm_grad_ctas(int64_t rows, int64_t hidden, int bf16, int sms, cudaError_t* err);
int norm_grad_partials(int64_t rows, int64_t hidden, int sms, int ctas);
// *partial_rows: rows of partial sums that it leaves
cudaError_t launch_norm_grad(const NormParams& p, int bf16, int ctas, cudaStream_t stream, int pdl,
                             int* partial_rows);

// --------------------------------------------- gradient of an activation, bias
struct DactParams {
  int32_t rows, cols;
  int32_t act;
  int32_t chunk_rows;   // rows of a CTA
  const void* d_out;
  const void* z;
  void* d_z;
  float* partials;      // [chunks][cols]
};

cudaError_t launch_dact(const DactParams& p, int bf16, int chunks, cudaStream_t stream, int pdl);
// chunks of rows for the kernel above, on so many SMs
int dact_chunks(int64_t rows, int64_t cols, int sms);

// out[c] = the sum of partials[r][c], rows in a fixed order
cudaError_t launch_column_sums(const float* partials, int rows, int cols, float* out,
                               cudaStream_t stream, int pdl);

// a launch that may overlap its set-up with the kernel before it (programmatic
// stream serialisation), unless `pdl` is 0
template <typename... Formal, typename... Actual>
cudaError_t launch_pdl(void (*kernel)(Formal...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t stream, int pdl, const Actual&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace gf
