// Host entry points of expert routing and of the e4m3 quantiser: checks of the
// arguments, the plan's chunks, launches.
#include <cuda_runtime.h>
#include <stdint.h>

#include "gf.h"
#include "moe.h"
#include "params.h"
#include "plan.h"
#include "runtime_internal.h"

namespace {

using gf::runtime_fail;

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxHidden = int64_t(1) << 24;  // columns are int32 in the kernels

bool given(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// scales are read and written one at a time: a part of a larger array will do
bool given_scale(const void* p) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0;
}

// Up to these sizes one kernel sorts and copies: every CTA counts all slots alone
// and copies its own tokens' rows. Above, the copies have a kernel of their own,
// whose CTAs the hardware balances. us, one kernel and two (16-bit rows; e4m3):
//   1024 tokens, 8 slots, 1024 columns    7.1  16.5     6.2  12.4
//   4096, 8, 1024                        18.6  24.6    14.3  15.7
//   2048, 8, 2048                        17.5  23.9    12.8  15.1
//   4096, 8, 2048                        32.7  30.1    22.2  19.7
//   2048, 8, 4096                        31.4  30.0    20.9  19.4
//   4096, 8, 64                           7.7  11.1     9.1  14.4
//   16384, 8, 64                         21.7  17.5    25.7  22.0
constexpr int64_t kFusedSlots = 49152, kFusedElements = 40 << 20;

// Whether clusters of CTAs share the counting of a sort without copies in it, which
// is worth the more the more slots there are, and the less the more experts. us, each
// CTA alone and clusters: 32768 slots of 128 experts 6.4 and 8.0, 65536 9.9 and 9.5,
// 65536 of 1024 experts 10.4 and 16.9. With the copies after it, which wait for the
// sort's last CTA, from fewer slots on (8 slots a token, 4096 columns):
//   experts   20480 slots    32768          49152          65536
//   128       35.0  35.0     52.6  53.0     76.8  74.5     102.7  96.7
//   256       35.1  35.3     53.0  54.0     78.0  75.1     103.2  97.3
//   512       35.2  37.1     52.2  52.7     76.4  76.2     101.8  98.6
//   1024      35.2  40.4     52.4  55.6     77.9  76.9     102.3 100.2
bool clusters_count(int64_t slots, int64_t experts, bool copies) {
  return slots > (copies ? 24576 + 32 * experts : 49152 + 64 * experts);
}

// Tokens of a chunk. One chunk per SM; smaller ones of kMoeChunkSlots slots where those
// are at most two an SM, of which one ranks its slots while the other still counts.
// More must not be: every CTA, or every cluster of them, counts all slots, and the
// sort would be quadratic. us, chunks of 4096 slots and one per SM: 800000 slots of
// 128 experts 32.7 and 36.4, 1 Mi 37.6 and 45.1, 1600000 76 and 65, 8 Mi of 256
// experts 1169 and 325. Where the copies are in the same launch the kernel's table
// holds kMoeChunkSlots rows.
int64_t chunk_of(int64_t tokens, int64_t topk, int sms, bool fused) {
  const int64_t per_sm = (tokens + sms - 1) / sms, small = gf::kMoeChunkSlots / topk;
  const bool few = fused || (tokens + small - 1) / small <= 2 * sms;
  const int64_t chunk = few && small < per_sm ? small : per_sm;
  return chunk < 1 ? 1 : chunk;
}

bool is_moe(const gf_plan* p) { return p != nullptr && p->epi == gf::EPI_MOE; }

gf_status dispatch(const gf_plan* p, const int32_t* expert, const void* x, int32_t* offsets,
                   int32_t* row_of, int32_t* slot_of, void* rows, float* scale, int copy,
                   cudaStream_t st) {
  const bool some = p->m > 0;
  if (!given(offsets)) return runtime_fail(GF_ERR_INVALID_VALUE);
  if (some && (!given(expert) || !given(row_of) || !given(slot_of)))
    return runtime_fail(GF_ERR_INVALID_VALUE);
  if (some && copy != gf::MOE_SORT_ONLY && (!given(x) || !given(rows)))
    return runtime_fail(GF_ERR_INVALID_VALUE);
  if (some && copy == gf::MOE_COPY_FP8 && !given_scale(scale)) return runtime_fail(GF_ERR_INVALID_VALUE);
  if (cudaSetDevice(p->device) != cudaSuccess) return runtime_fail(GF_ERR_CUDA);
  gf::MoeParams prm = {};
  prm.tokens = static_cast<int32_t>(p->m);
  prm.topk = static_cast<int32_t>(p->topk);
  prm.experts = static_cast<int32_t>(p->experts);
  prm.hidden = static_cast<int32_t>(p->k);
  prm.slots = static_cast<int32_t>(p->m * p->topk);
  prm.chunk_tokens = p->chunk_tokens;
  prm.num_chunks = p->num_chunks;
  const bool copies = copy != gf::MOE_SORT_ONLY;
  prm.clusters = !(copies && p->fused) && clusters_count(prm.slots, p->experts, copies) ? 1 : 0;
  prm.fused = p->fused;
  prm.expert = expert;
  prm.offsets = offsets;
  prm.row_of = row_of;
  prm.slot_of = slot_of;
  prm.x = x;
  prm.rows = rows;
  prm.scale = scale;
  // CTAs that share a chunk's copies: one per 8 Ki elements of its rows, as far as
  // there are SMs for them (an SM holds one). One token, 8 slots, 16384 columns 6.2
  // us, with one CTA 8.3; 65536 columns 6.3 and 20.6
  const int64_t items = p->chunk_tokens * ((p->k + 511) / 512);
  int64_t seg = (items + 15) / 16;
  const int64_t room = p->num_sms / p->num_chunks;
  seg = seg > room ? room : seg;
  prm.segments = static_cast<int32_t>(seg < 1 ? 1 : seg);
  const int bf16 = p->dtype == GF_BF16 ? 1 : 0;
  if (gf::launch_moe_dispatch(prm, copy, bf16, st, p->pdl) != cudaSuccess)
    return runtime_fail(GF_ERR_CUDA);
  return GF_OK;
}

gf::GatherParams gather_params(const gf_plan* p, const int32_t* row_of, const float* weight,
                               const void* rows, void* out) {
  gf::GatherParams g = {};
  g.tokens = static_cast<int32_t>(p->m);
  g.topk = static_cast<int32_t>(p->topk);
  g.hidden = static_cast<int32_t>(p->k);
  g.slots = static_cast<int32_t>(p->m * p->topk);
  g.experts = static_cast<int32_t>(p->experts);
  g.row_of = row_of;
  g.weight = weight;
  g.rows = rows;
  g.out = out;
  return g;
}

}  // namespace

extern "C" {

GF_API gf_plan* gf_moe_plan(int64_t tokens, int64_t topk, int64_t experts, int64_t hidden,
                            gf_dtype dtype) {
  if (tokens < 0 || tokens > kMaxDim || topk < 1 || topk > 64 || experts < 1 ||
      experts > gf::kMaxExperts || hidden < 1 || hidden > kMaxHidden ||
      tokens * topk > kMaxDim || (dtype != GF_F16 && dtype != GF_BF16)) {
    runtime_fail(GF_ERR_INVALID_VALUE);
    return nullptr;
  }
  int dev = 0, sms = 0;
  const gf_status st = gf::runtime_device(&dev, &sms);
  if (st != GF_OK) {
    runtime_fail(st);
    return nullptr;
  }
  const int fused = tokens * topk <= kFusedSlots && tokens * topk * hidden <= kFusedElements ? 1 : 0;
  const int64_t chunk = chunk_of(tokens, topk, sms, fused != 0);
  const int64_t chunks = tokens == 0 ? 1 : (tokens + chunk - 1) / chunk;
  gf_plan* p = gf::runtime_new_plan(gf::EPI_MOE, dtype);
  if (!p) return nullptr;
  p->m = tokens;
  p->k = hidden;
  p->n = experts;
  p->topk = topk;
  p->experts = experts;
  p->chunk_tokens = static_cast<int>(chunk);
  p->num_chunks = static_cast<int>(chunks);
  p->fused = fused;
  p->grid = static_cast<int>(chunks);
  return p;
}

GF_API gf_status gf_moe_dispatch_execute(const gf_plan* p, const int32_t* expert, const void* x,
                                         int32_t* offsets, int32_t* row_of, int32_t* slot_of,
                                         void* rows, struct CUstream_st* stream) {
  if (!is_moe(p)) return runtime_fail(GF_ERR_INVALID_VALUE);
  const int copy = x == nullptr && rows == nullptr ? gf::MOE_SORT_ONLY : gf::MOE_COPY;
  return dispatch(p, expert, x, offsets, row_of, slot_of, rows, nullptr, copy,
                  reinterpret_cast<cudaStream_t>(stream));
}

GF_API gf_status gf_moe_dispatch_fp8_execute(const gf_plan* p, const int32_t* expert,
                                             const void* x, int32_t* offsets, int32_t* row_of,
                                             int32_t* slot_of, void* rows, float* scale,
                                             struct CUstream_st* stream) {
  if (!is_moe(p)) return runtime_fail(GF_ERR_INVALID_VALUE);
  if (p->k % 16 != 0) return runtime_fail(GF_ERR_UNSUPPORTED);
  return dispatch(p, expert, x, offsets, row_of, slot_of, rows, scale, gf::MOE_COPY_FP8,
                  reinterpret_cast<cudaStream_t>(stream));
}

GF_API gf_status gf_moe_dispatch_grad_execute(const gf_plan* p, const int32_t* row_of,
                                              const void* d_rows, void* d_x,
                                              struct CUstream_st* stream) {
  if (!is_moe(p)) return runtime_fail(GF_ERR_INVALID_VALUE);
  if (p->m == 0) return GF_OK;
  if (!given(row_of) || !given(d_rows) || !given(d_x)) return runtime_fail(GF_ERR_INVALID_VALUE);
  if (cudaSetDevice(p->device) != cudaSuccess) return runtime_fail(GF_ERR_CUDA);
  const gf::GatherParams g = gather_params(p, row_of, nullptr, d_rows, d_x);
  return gf::launch_moe_gather(g, p->dtype == GF_BF16, p->num_sms,
                               reinterpret_cast<cudaStream_t>(stream), p->pdl) == cudaSuccess
             ? GF_OK
             : runtime_fail(GF_ERR_CUDA);
}

GF_API gf_status gf_moe_combine_execute(const gf_plan* p, const int32_t* row_of,
                                        const float* weight, const void* rows, void* out,
                                        struct CUstream_st* stream) {
  if (!is_moe(p)) return runtime_fail(GF_ERR_INVALID_VALUE);
  if (p->m == 0) return GF_OK;
  if (!given(row_of) || !given(weight) || !given(rows) || !given(out))
    return runtime_fail(GF_ERR_INVALID_VALUE);
  if (cudaSetDevice(p->device) != cudaSuccess) return runtime_fail(GF_ERR_CUDA);
  const gf::GatherParams g = gather_params(p, row_of, weight, rows, out);
  return gf::launch_moe_gather(g, p->dtype == GF_BF16, p->num_sms,
                               reinterpret_cast<cudaStream_t>(stream), p->pdl) == cudaSuccess
             ? GF_OK
             : runtime_fail(GF_ERR_CUDA);
}

GF_API gf_status gf_moe_combine_grad_execute(const gf_plan* p, const int32_t* offsets,
                                             const int32_t* row_of, const float* weight,
                                             const void* rows, const void* d_out, void* d_rows,
                                             float* d_weight, struct CUstream_st* stream) {
  if (!is_moe(p)) return runtime_fail(GF_ERR_INVALID_VALUE);
  if (p->m == 0) return GF_OK;
  if (!given(offsets) || !given(row_of) || !given(weight) || !given(rows) || !given(d_out) ||
      !given(d_rows) || !given(d_weight))
    return runtime_fail(GF_ERR_INVALID_VALUE);
  if (cudaSetDevice(p->device) != cudaSuccess) return runtime_fail(GF_ERR_CUDA);
  gf::GatherParams g = gather_params(p, row_of, weight, rows, d_rows);
  g.offsets = offsets;
  g.d_out = d_out;
  g.d_weight = d_weight;
  return gf::launch_moe_combine_grad(g, p->dtype == GF_BF16,
                                     reinterpret_cast<cudaStream_t>(stream),
                                     p->pdl) == cudaSuccess
             ? GF_OK
             : runtime_fail(GF_ERR_CUDA);
}

GF_API gf_status gf_fp8_quantize(int64_t m, int64_t k, gf_dtype dtype, int32_t block_rows,
                                 const void* x, void* q, float* scale,
                                 struct CUstream_st* stream) {
  if (m < 0 || k < 0 || m > kMaxDim || k > kMaxDim || (dtype != GF_F16 && dtype != GF_BF16) ||
      (block_rows != 1 && block_rows != 128))
    return runtime_fail(GF_ERR_INVALID_VALUE);
  if (k % 16 != 0) return runtime_fail(GF_ERR_UNSUPPORTED);
  // one CTA per 128 x 128 block, or per 64 blocks of 1 x 128
  const int64_t blocks_k = (k + 127) / 128;
  if ((block_rows == 128 ? (m + 127) / 128 * blocks_k : m * blocks_k / 64 + 1) > kMaxDim)
    return runtime_fail(GF_ERR_UNSUPPORTED);
  const bool empty = m == 0 || k == 0;
  if (!empty && (!given(x) || !given(q) || !given_scale(scale)))
    return runtime_fail(GF_ERR_INVALID_VALUE);
  int dev = 0, sms = 0;
  const gf_status st = gf::runtime_device(&dev, &sms);
  if (st != GF_OK) return runtime_fail(st);
  if (empty) return GF_OK;
  if (cudaSetDevice(dev) != cudaSuccess) return runtime_fail(GF_ERR_CUDA);
  return gf::launch_fp8_quantize(m, k, dtype == GF_BF16, block_rows, x, q, scale,
                                 reinterpret_cast<cudaStream_t>(stream), 1) == cudaSuccess
             ? GF_OK
             : runtime_fail(GF_ERR_CUDA);
}

}  // extern "C"
