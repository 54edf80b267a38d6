// Host-side view of the expert-routing and quantising kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gf {

constexpr int kMaxExperts = 1024;
// most slots of a chunk that is sorted and copied in one launch: their rows are held
// in shared memory
constexpr int kMoeChunkSlots = 4096;

struct MoeParams {
  int32_t tokens, topk, experts;
  int32_t hidden;
  int32_t slots;         // tokens * topk
  int32_t chunk_tokens;  // tokens per CTA of the sort
  int32_t num_chunks;
  int32_t clusters;      // 1: clusters of CTAs share the counting; 0: every CTA counts alone
  int32_t fused;         // 1: the sort kernel copies too
  int32_t segments;      // CTAs that share the copies of one chunk (along hidden)
  const int32_t* expert;
  int32_t* offsets;
  int32_t* row_of;
  int32_t* slot_of;
  const void* x;
  void* rows;
  float* scale;
};

enum MoeCopy : int { MOE_SORT_ONLY = 0, MOE_COPY = 1, MOE_COPY_FP8 = 2 };

cudaError_t launch_moe_dispatch(const MoeParams& p, int copy, int bf16, cudaStream_t stream,
                                int pdl);

struct GatherParams {
  int32_t tokens, topk;
  int32_t hidden;
  int32_t slots;
  const int32_t* offsets;  // gradient: its entry `experts` bounds the rows with a slot
  int32_t experts;
  const int32_t* row_of;
  const float* weight;     // NULL: ones
  const void* rows;
  const void* d_out;
  void* out;               // forward: [tokens, hidden]; gradient: d_rows
  float* d_weight;
};

cudaError_t launch_moe_gather(const GatherParams& p, int bf16, int sms, cudaStream_t stream,
                              int pdl);
cudaError_t launch_moe_combine_grad(const GatherParams& p, int bf16, cudaStream_t stream,
                                    int pdl);

cudaError_t launch_fp8_quantize(int64_t m, int64_t k, int bf16, int block_rows, const void* x,
                                void* q, float* scale, cudaStream_t stream, int pdl);

}  // namespace gf
