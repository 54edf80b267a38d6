// Host entry points of the router, the root-mean-square norm and the gradient of
// an activation and its bias: checks of the arguments, plans, launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "block.h"
#include "gf.h"
#include "moe.h"
#include "params.h"
#include "plan.h"
#include "runtime_internal.h"

namespace {

using gf::runtime_fail;

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxLd = int64_t(1) << 24;  // elements between rows of logits

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool given(const void* p) { return p != nullptr && aligned(p); }
// read or written one fp32 value at a time: a part of a larger array will do
bool given_f32(const void* p) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0;
}

bool is_plan(const gf_plan* p, int epi) { return p != nullptr && p->epi == epi; }

gf_status launched(cudaError_t e) { return e == cudaSuccess ? GF_OK : runtime_fail(GF_ERR_CUDA); }

gf_plan* refuse(gf_status s) {
  runtime_fail(s);
  return nullptr;
}

bool known_act(int act) { return act >= GF_ACT_NONE && act <= GF_ACT_SILU; }

// The fp32 column sums of a backward pass, one row for each CTA or chunk.
gf_status add_partials(gf_plan* p, int64_t rows, int64_t cols) {
  const size_t bytes = static_cast<size_t>(rows) * static_cast<size_t>(cols) * 4;
  if (bytes == 0) return GF_OK;
  if (cudaMalloc(&p->d_work, bytes) != cudaSuccess) {
    cudaGetLastError();
    p->d_work = nullptr;
    return GF_ERR_OUT_OF_MEMORY;
  }
  p->work_bytes = bytes;
  return GF_OK;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------- router
static gf::RouteParams route_params(const gf_plan* p, const void* logits) {
  gf::RouteParams r = {};
  r.tokens = static_cast<int32_t>(p->m);
  r.experts = static_cast<int32_t>(p->experts);
  r.topk = static_cast<int32_t>(p->topk);
  r.groups = static_cast<int32_t>(p->groups);
  r.group_size = static_cast<int32_t>(p->experts / p->groups);
  r.topk_groups = static_cast<int32_t>(p->topk_groups);
  r.group_best = p->group_best;
  r.sigmoid = p->score == GF_SCORE_SIGMOID ? 1 : 0;
  r.renorm = p->renorm;
  r.scale = p->scale;
  r.ld = p->ld;
  r.logits = logits;
  r.sms = p->num_sms;
  return r;
}

static int logits_type(const gf_plan* p) {
  return p->dtype == GF_F32 ? 2 : p->dtype == GF_BF16 ? 1 : 0;
}

GF_API gf_plan* gf_route_plan(int64_t tokens, int64_t experts, int64_t topk, gf_dtype dtype,
                              gf_score score, int32_t renorm, float scale, int64_t groups,
                              int64_t topk_groups, int32_t group_best, int64_t ld) {
  if (tokens < 0 || tokens > kMaxDim || experts < 1 || experts > gf::kMaxExperts || topk < 1 ||
      topk > 64 || tokens * topk > kMaxDim || (dtype != GF_F16 && dtype != GF_BF16 && dtype != GF_F32) ||
      (score != GF_SCORE_SOFTMAX && score != GF_SCORE_SIGMOID) || (renorm != 0 && renorm != 1) ||
      !isfinite(scale) || groups < 1 || groups > experts || topk_groups < 1 ||
      topk_groups > groups || (group_best != 1 && group_best != 2) || ld < experts || ld > kMaxLd)
    return refuse(GF_ERR_INVALID_VALUE);
  if (experts % groups != 0 || topk > experts / groups * topk_groups)
    return refuse(GF_ERR_INVALID_VALUE);
  if (groups > gf::kRouteMaxGroups) return refuse(GF_ERR_UNSUPPORTED);
  gf_plan* p = gf::runtime_new_plan(gf::EPI_ROUTE, dtype);
  if (!p) return nullptr;
  p->m = tokens;
  p->n = experts;
  p->topk = topk;
  p->experts = experts;
  p->groups = groups;
  p->topk_groups = topk_groups;
  p->group_best = group_best;
  p->ld = ld;
  p->score = score;
  p->renorm = renorm;
  p->scale = scale;
  p->tile_n = static_cast<int>(experts);
  p->grid = static_cast<int>(gf::route_ctas(route_params(p, nullptr), logits_type(p), &p->tile_rows));
  return p;
}

GF_API gf_status gf_route_execute(const gf_plan* p, const void* logits, const float* bias,
                                  int32_t* expert, float* weight, struct CUstream_st* stream) {
  if (!is_plan(p, gf::EPI_ROUTE)) return runtime_fail(GF_ERR_INVALID_VALUE);
  if (p->m == 0) return GF_OK;
  if (!given(logits) || !given(expert) || !given(weight) || (bias != nullptr && !given_f32(bias)))
    return runtime_fail(GF_ERR_INVALID_VALUE);
  if (cudaSetDevice(p->device) != cudaSuccess) return runtime_fail(GF_ERR_CUDA);
  gf::RouteParams r = route_params(p, logits);
  r.bias = bias;
  r.expert = expert;
  r.weight = weight;
  return launched(gf::launch_route(r, logits_type(p), reinterpret_cast<cudaStream_t>(stream), p->pdl));
}

GF_API gf_status gf_route_grad_execute(const gf_plan* p, const void* logits, const int32_t* expert,
                                       const float* d_weight, void* d_logits,
                                       struct CUstream_st* stream) {
  if (!is_plan(p, gf::EPI_ROUTE)) return runtime_fail(GF_ERR_INVALID_VALUE);
  if (p->m == 0) return GF_OK;
  if (!given(logits) || !given(expert) || !given(d_weight) || !given(d_logits))
    return runtime_fail(GF_ERR_INVALID_VALUE);
  if (cudaSetDevice(p->device) != cudaSuccess) return runtime_fail(GF_ERR_CUDA);
  gf::RouteParams r = route_params(p, logits);
  r.expert = const_cast<int32_t*>(expert);
  r.d_weight = d_weight;
  r.d_logits = d_logits;
  return launched(gf::launch_route_grad(r, logits_type(p), reinterpret_cast<cudaStream_t>(stream), p->pdl));
}

// --------------------------------------------------------------------- norm
static gf::NormParams norm_params(const gf_plan* p) {
  gf::NormParams n = {};
  n.rows = static_cast<int32_t>(p->m);
  n.hidden = static_cast<int32_t>(p->n);
  n.eps = p->scale;
  n.sms = p->num_sms;
  n.status = p->d_status;
  n.wait_limit_ns = p->wait_limit_ns;
  n.drop_load = p->drop_load;
  return n;
}

GF_API gf_plan* gf_rmsnorm_plan(int64_t rows, int64_t hidden, gf_dtype dtype, float eps) {
  if (rows < 0 || rows > kMaxDim || hidden < 1 || hidden > kMaxDim ||
      (dtype != GF_F16 && dtype != GF_BF16) || !(eps >= 0.f) || !isfinite(eps))
    return refuse(GF_ERR_INVALID_VALUE);
  if (hidden > gf::kNormMaxHidden) return refuse(GF_ERR_UNSUPPORTED);
  gf_plan* p = gf::runtime_new_plan(gf::EPI_NORM, dtype);
  if (!p) return nullptr;
  p->m = rows;
  p->n = p->k = hidden;
  p->scale = eps;
  p->tile_n = static_cast<int>(hidden);
  p->grid = static_cast<int>(gf::norm_ctas(norm_params(p), &p->tile_rows, &p->stages));
  return p;
}

// What the gradient alone needs, made by the first call that does: the CTAs of the kernel that
// loads its rows itself and, for d_weight, the workspace. That call may be captured into a graph:
// the relaxed mode lets this thread allocate meanwhile.
static gf_status norm_grad_ready(gf_plan* p, bool sums) {
  std::lock_guard<std::mutex> lock(p->cache_mu);
  if (p->num_chunks == 0) {
    cudaError_t e = cudaSuccess;
    p->num_chunks = gf::norm_grad_ctas(p->m, p->n, p->dtype == GF_BF16, p->num_sms, &e);
    if (e != cudaSuccess) {
      cudaGetLastError();
      p->num_chunks = 0;
      return GF_ERR_CUDA;
    }
  }
  if (!sums || p->d_work != nullptr) return GF_OK;
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return GF_ERR_CUDA;
  const gf_status st =
      add_partials(p, gf::norm_grad_partials(p->m, p->n, p->num_sms, p->num_chunks), p->n);
  cudaThreadExchangeStreamCaptureMode(&mode);
  return st;
}

GF_API gf_status gf_rmsnorm_execute(const gf_plan* p, const void* x, const void* residual,
                                    const void* weight, void* residual_out, void* out, void* out8,
                                    float* out_scale, struct CUstream_st* stream) {
  if (!is_plan(p, gf::EPI_NORM)) return runtime_fail(GF_ERR_INVALID_VALUE);
  if (p->m == 0) return GF_OK;
  if (!given(x) || !given(weight) || !aligned(residual) || !aligned(residual_out) || !aligned(out) ||
      !aligned(out8))
    return runtime_fail(GF_ERR_INVALID_VALUE);
  if ((out == nullptr && out8 == nullptr) || (residual == nullptr && residual_out != nullptr) ||
      (out8 == nullptr) != (out_scale == nullptr) || (out8 != nullptr && !given_f32(out_scale)))
    return runtime_fail(GF_ERR_INVALID_VALUE);
  if (out8 != nullptr && p->n % 16 != 0) return runtime_fail(GF_ERR_UNSUPPORTED);
  if (cudaSetDevice(p->device) != cudaSuccess) return runtime_fail(GF_ERR_CUDA);
  gf::NormParams n = norm_params(p);
  n.x = x;
  n.residual = residual;
  n.weight = weight;
  n.residual_out = residual_out;
  n.out = out;
  n.out8 = static_cast<uint8_t*>(out8);
  n.scale = out_scale;
  return launched(gf::launch_norm(n, p->dtype == GF_BF16, reinterpret_cast<cudaStream_t>(stream), p->pdl));
}

GF_API gf_status gf_rmsnorm_grad_execute(const gf_plan* p, const void* d_out, const void* r,
                                         const void* weight, const void* d_residual, void* d_x,
                                         float* d_weight, struct CUstream_st* stream) {
  if (!is_plan(p, gf::EPI_NORM)) return runtime_fail(GF_ERR_INVALID_VALUE);
  if (d_weight != nullptr && !given_f32(d_weight)) return runtime_fail(GF_ERR_INVALID_VALUE);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (p->m == 0) {
    // the sum over no rows
    if (d_weight == nullptr) return GF_OK;
    if (cudaSetDevice(p->device) != cudaSuccess) return runtime_fail(GF_ERR_CUDA);
    return launched(cudaMemsetAsync(d_weight, 0, static_cast<size_t>(p->n) * 4, st));
  }
  if (!given(d_out) || !given(r) || !given(weight) || !aligned(d_residual) || !given(d_x))
    return runtime_fail(GF_ERR_INVALID_VALUE);
  if (cudaSetDevice(p->device) != cudaSuccess) return runtime_fail(GF_ERR_CUDA);
  const gf_status ready = norm_grad_ready(const_cast<gf_plan*>(p), d_weight != nullptr);
  if (ready != GF_OK) return runtime_fail(ready);
  gf::NormParams n = norm_params(p);
  n.x = r;
  n.residual = d_residual;
  n.weight = weight;
  n.out = d_x;
  n.d_out = d_out;
  n.partials = d_weight != nullptr ? static_cast<float*>(p->d_work) : nullptr;
  int partial_rows = 0;
  cudaError_t e = gf::launch_norm_grad(n, p->dtype == GF_BF16, p->num_chunks, st, p->pdl, &partial_rows);
  if (e == cudaSuccess && d_weight != nullptr)
    e = gf::launch_column_sums(n.partials, partial_rows, n.hidden, d_weight, st, p->pdl);
  return launched(e);
}

// --------------------------------------------- gradient of an activation, bias
GF_API gf_plan* gf_dact_bgrad_plan(int64_t m, int64_t n, gf_dtype dtype, gf_activation act) {
  if (m < 0 || n < 0 || m > kMaxDim || n > kMaxDim || (dtype != GF_F16 && dtype != GF_BF16) ||
      !known_act(act))
    return refuse(GF_ERR_INVALID_VALUE);
  if (n % 8 != 0) return refuse(GF_ERR_UNSUPPORTED);
  gf_plan* p = gf::runtime_new_plan(gf::EPI_DACT, dtype);
  if (!p) return nullptr;
  p->m = m;
  p->n = n;
  p->act = act;
  p->num_chunks = m == 0 || n == 0 ? 0 : gf::dact_chunks(m, n, p->num_sms);
  p->tile_rows = p->num_chunks == 0 ? 0 : static_cast<int>((m + p->num_chunks - 1) / p->num_chunks);
  p->tile_n = 256;
  const int64_t ctas = (n + 255) / 256 * p->num_chunks;
  p->grid = static_cast<int>(ctas < kMaxDim ? ctas : kMaxDim);
  const gf_status st = add_partials(p, p->num_chunks, n);
  if (st != GF_OK) {
    gf_plan_free(p);
    return refuse(st);
  }
  return p;
}

GF_API gf_status gf_dact_bgrad_execute(const gf_plan* p, const void* d_out, const void* z, void* d_z,
                                       float* bgrad, struct CUstream_st* stream) {
  if (!is_plan(p, gf::EPI_DACT)) return runtime_fail(GF_ERR_INVALID_VALUE);
  if (bgrad != nullptr && !given_f32(bgrad)) return runtime_fail(GF_ERR_INVALID_VALUE);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (p->m == 0 || p->n == 0) {
    if (bgrad == nullptr || p->n == 0) return GF_OK;
    if (cudaSetDevice(p->device) != cudaSuccess) return runtime_fail(GF_ERR_CUDA);
    return launched(cudaMemsetAsync(bgrad, 0, static_cast<size_t>(p->n) * 4, st));
  }
  // without an activation d_z is d_out, and only the bias has something to form
  const bool plain = p->act == GF_ACT_NONE;
  if (!given(d_out) || (plain ? z != nullptr || d_z != nullptr || bgrad == nullptr
                              : !given(z) || !given(d_z)))
    return runtime_fail(GF_ERR_INVALID_VALUE);
  if (cudaSetDevice(p->device) != cudaSuccess) return runtime_fail(GF_ERR_CUDA);
  gf::DactParams d = {};
  d.rows = static_cast<int32_t>(p->m);
  d.cols = static_cast<int32_t>(p->n);
  d.act = p->act;
  d.chunk_rows = p->tile_rows;
  d.d_out = d_out;
  d.z = z;
  d.d_z = d_z;
  d.partials = bgrad != nullptr ? static_cast<float*>(p->d_work) : nullptr;
  cudaError_t e = gf::launch_dact(d, p->dtype == GF_BF16, p->num_chunks, st, p->pdl);
  if (e == cudaSuccess && bgrad != nullptr)
    e = gf::launch_column_sums(d.partials, p->num_chunks, d.cols, bgrad, st, p->pdl);
  return launched(e);
}

}  // extern "C"
