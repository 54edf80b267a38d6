// Host entry points of the block-scaled e4m3 products: checks of the
// arguments, the plan's tiles, tensor maps and launch.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <cmath>

#include "fp8_params.h"
#include "gf.h"
#include "params.h"
#include "plan.h"
#include "runtime_internal.h"

namespace {

using gf::runtime_fail;

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

bool given(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// scales are read and written one at a time: a part of a larger array will do
bool given_scale(const void* p) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0;
}

// GF_OPT_KERNEL
enum : int { kNarrow16 = 1, kNarrow64 = 2, kSingle = 3, kPair = 4 };

// What a kernel takes, in us: start + block * (k-blocks one after the other on
// an SM) + round * (tiles one after the other on it). Fitted to the times of all four
// for 526 products (8 to 51200 rows, 1 to 128 groups, 256 to 17408 columns, k 512
// to 16384). The kernel that it names is within 1 % of the best of the four on
// average and 37 % at worst (256 rows, 256 columns, k = 16384: 64-row tiles 18.3
// us, 16-row tiles 13.4). Some of them (rows, columns, k; "64 x": groups):
//                           16-row  64-row  single  pair
//   8, 17408, 8192            26      32      40     45
//   48, 9000, 8192            30      20      32     29
//   256, 4096, 8192           55      22      31     28
//   256, 17408, 8192         196      77      38     36
//   64 x 64, 4096, 2048        -     119      90    130
//   64 x 256, 4096, 2048       -     353     161    181
//   8 x 1024, 4096, 16384      -       -     482    425
struct Pace {
  double start, block, round;
};
constexpr Pace kPace[2][4] = {
    // 16-row tiles, 64-row tiles, single CTA, CTA pair
    {{4.0, 0.22, 0.8}, {4.0, 0.29, 1.2}, {3.4, 0.38, 2.8}, {4.2, 0.34, 2.8}},
    {{4.0, 0.32, 3.0}, {4.0, 0.75, 7.0}, {4.6, 0.35, 3.0}, {4.8, 0.33, 3.6}}};  // SwiGLU

// The time of one kernel for the plan. The rows of each group are on the
// device: they are taken to be about alike, with a part of a tile more each.
double expected_time(const gf_plan* p, int kernel) {
  const int dual = p->epi == gf::EPI_FP8_SWIGLU_QUANT ? 1 : 0;
  const int64_t tile_rows = kernel == kNarrow16 ? 16 : kernel == kNarrow64 ? 64
                            : kernel == kSingle ? 128 : 256;
  const int64_t tile_n = kernel <= kNarrow64 || dual ? 128 : 256;
  const double groups = static_cast<double>(p->groups), m = static_cast<double>(p->m);
  const double row_tiles = p->groups == 1 ? std::ceil(m / tile_rows)
                                          : groups * std::max(1.0, m / groups / tile_rows + 0.4);
  const double tiles = row_tiles * static_cast<double>((p->n + tile_n - 1) / tile_n);
  const double each = tiles / (kernel == kPair ? p->max_pair_clusters : p->num_sms);
  const double rounds = p->groups == 1 ? std::ceil(each) : std::max(1.0, each);
  const double kb = static_cast<double>((p->k + 127) / 128);
  double blocks = rounds * kb;
  const double whole = std::ceil(each);
  if (kernel <= kNarrow64 && 100 * each < gf::fp8_whole_fill(whole > 1 ? 2 : 1) * whole)
    blocks = std::min(blocks, each * kb +
                                  gf::fp8_join_blocks(static_cast<int>(tile_rows), dual));
  const Pace& c = kPace[dual][kernel - 1];
  return c.start + c.block * blocks + c.round * rounds;
}

// Kernel and tiles of the plan.
void plan_tiles(gf_plan* p) {
  const int dual = p->epi == gf::EPI_FP8_SWIGLU_QUANT ? 1 : 0;
  const int tile_n = dual ? 128 : 256;  // of the single-CTA and the pair kernel
  int kernel = p->forced_kernel;
  if (kernel == 0) {
    kernel = kNarrow16;
    for (int other = kNarrow64; other <= (p->max_pair_clusters > 0 ? kPair : kSingle); ++other)
      if (expected_time(p, other) < expected_time(p, kernel)) kernel = other;
  }
  if (kernel == kPair && p->max_pair_clusters == 0) kernel = kSingle;
  p->kernel = kernel;
  p->tile_n = kernel <= kNarrow64 ? 128 : tile_n;
  p->grid = kernel == kPair ? 2 * p->max_pair_clusters : p->num_sms;
  p->tile_rows = kernel == kNarrow16 ? 16 : kernel == kNarrow64 ? 64 : kernel == kSingle ? 128 : 256;
  p->stages = kernel == kPair     ? gf::fp8_wide_stages()
              : kernel == kSingle ? gf::fp8_single_stages()
                                  : gf::fp8_narrow_stages(p->tile_rows, dual);
}

// The workspace of the plan's tiling: the narrow kernel's counters (zeroed),
// then its partial sums. Grown when too small; one that the plan has already
// had may be in use, by launches that have to end first.
size_t counter_bytes(const gf_plan* p) { return (static_cast<size_t>(p->grid) * 4 + 255) / 256 * 256; }

gf_status ensure_work(gf_plan* p) {
  if (p->kernel > kNarrow64) return GF_OK;
  const int dual = p->epi == gf::EPI_FP8_SWIGLU_QUANT ? 1 : 0;
  if (p->d_work && cudaDeviceSynchronize() != cudaSuccess) return GF_ERR_CUDA;
  const size_t need =
      counter_bytes(p) + gf::fp8_narrow_partial_bytes(p->tile_rows, dual, p->grid);
  if (need > p->work_bytes) {
    void* grown = nullptr;
    if (cudaMalloc(&grown, need) != cudaSuccess) {  // the plan keeps what it has
      cudaGetLastError();
      return GF_ERR_OUT_OF_MEMORY;
    }
    if (p->d_work) cudaFree(p->d_work);
    p->d_work = grown;
    p->work_bytes = need;
  }
  return gf::runtime_zero(p->d_work, counter_bytes(p));
}

}  // namespace

namespace gf {

gf_status runtime_fp8_set_kernel(gf_plan* p, int64_t value) {
  if (value < 0 || value > 4) return GF_ERR_INVALID_VALUE;
  if (value == 4 && p->max_pair_clusters == 0) return GF_ERR_UNSUPPORTED;
  if (cudaSetDevice(p->device) != cudaSuccess) return GF_ERR_CUDA;
  const int before = p->forced_kernel;
  p->forced_kernel = static_cast<int>(value);
  plan_tiles(p);
  const gf_status st = ensure_work(p);
  if (st != GF_OK) {  // back to the kernel whose workspace the plan has
    p->forced_kernel = before;
    plan_tiles(p);
  }
  return st;
}

int runtime_fp8_k_splits(const gf_plan* p) {
  if (p->kernel > kNarrow64) return 1;
  if (p->groups > 1) return 0;
  const int kb = static_cast<int>((p->k + 127) / 128);
  const int64_t tiles =
      kb == 0 ? 0 : (p->m + p->tile_rows - 1) / p->tile_rows * ((p->n + 127) / 128);
  const int ctas = fp8_split_ctas(static_cast<int>(tiles), kb, p->grid, p->tile_rows,
                                  p->epi == EPI_FP8_SWIGLU_QUANT ? 1 : 0);
  int most = 1;
  for (int64_t t = 0; ctas > 0 && t < tiles; ++t)
    most = std::max(most, fp8_unit_owner((t + 1) * kb - 1, tiles * kb, ctas) -
                              fp8_unit_owner(t * kb, tiles * kb, ctas) + 1);
  return most;
}

gf_status runtime_fp8_clear_counters(gf_plan* p) {
  if (p->kernel > kNarrow64) return GF_OK;
  return gf::runtime_zero(p->d_work, counter_bytes(p));
}

}  // namespace gf

extern "C" {

GF_API gf_plan* gf_fp8_matmul_plan(int64_t m, int64_t n, int64_t k, int64_t groups,
                                   gf_dtype dtype, gf_fp8_epilog epilog) {
  if (m < 0 || n < 0 || k < 0 || m > kMaxDim || n > kMaxDim || k > kMaxDim || groups < 1 ||
      groups > gf::kFp8MaxGroups || (dtype != GF_F16 && dtype != GF_BF16) ||
      (epilog != GF_FP8_EPILOG_NONE && epilog != GF_FP8_EPILOG_SWIGLU_QUANT)) {
    runtime_fail(GF_ERR_INVALID_VALUE);
    return nullptr;
  }
  const bool dual = epilog == GF_FP8_EPILOG_SWIGLU_QUANT;
  // the kernels count rows, rows of B over all groups and tiles (the smallest
  // are 16 rows x 128 columns) in int32, a tile or a round past the last one too
  if (k % 16 != 0 || n % (dual ? 16 : 8) != 0 || m > kMaxDim - 512 || groups * n > kMaxDim - 512 ||
      (m / 16 + groups + 1) * ((n + 127) / 128) > (int64_t(1) << 30)) {
    runtime_fail(GF_ERR_UNSUPPORTED);
    return nullptr;
  }
  gf_plan* p = gf::runtime_new_plan(dual ? gf::EPI_FP8_SWIGLU_QUANT : gf::EPI_FP8, dtype);
  if (!p) return nullptr;
  p->m = m;
  p->n = n;
  p->k = k;
  p->groups = groups;
  p->max_pair_clusters = gf::fp8_wide_max_clusters();
  cudaGetLastError();
  plan_tiles(p);
  const gf_status st = ensure_work(p);
  if (st != GF_OK) {
    gf_plan_free(p);
    runtime_fail(st);
    return nullptr;
  }
  return p;
}

GF_API gf_status gf_fp8_matmul_execute(const gf_plan* p, const void* A, const float* a_scale,
                                       const void* B, const float* b_scale, const void* B2,
                                       const float* b2_scale, const int32_t* offsets, void* out,
                                       float* out_scale, struct CUstream_st* stream) {
  if (!p || !gf::epi_fp8(p->epi)) return runtime_fail(GF_ERR_INVALID_VALUE);
  const bool dual = p->epi == gf::EPI_FP8_SWIGLU_QUANT;
  const bool empty = p->m == 0 || p->n == 0;
  if (!empty) {
    if (!given(out) || (dual && !given_scale(out_scale))) return runtime_fail(GF_ERR_INVALID_VALUE);
    if (p->k > 0 && (!given(A) || !given_scale(a_scale) || !given(B) || !given_scale(b_scale)))
      return runtime_fail(GF_ERR_INVALID_VALUE);
    if (p->k > 0 && dual && (!given(B2) || !given_scale(b2_scale)))
      return runtime_fail(GF_ERR_INVALID_VALUE);
    if (offsets == nullptr ? p->groups != 1 : !given(offsets))
      return runtime_fail(GF_ERR_INVALID_VALUE);
  }
  if (cudaSetDevice(p->device) != cudaSuccess) return runtime_fail(GF_ERR_CUDA);
  if (empty) return GF_OK;

  CUtensorMap tmA, tmB, tmB2;
  memset(&tmA, 0, sizeof tmA);
  memset(&tmB, 0, sizeof tmB);
  memset(&tmB2, 0, sizeof tmB2);
  if (p->k > 0) {
    const uint64_t b_rows = static_cast<uint64_t>(p->groups) * p->n;
    if (!gf::runtime_encode_2d_u8(&tmA, A, p->k, p->m, 128,
                                  p->tile_rows < 128 ? p->tile_rows : 128) ||
        !gf::runtime_encode_2d_u8(&tmB, B, p->k, b_rows, 128, 128) ||
        (dual && !gf::runtime_encode_2d_u8(&tmB2, B2, p->k, b_rows, 128, 128)))
      return runtime_fail(GF_ERR_INVALID_VALUE);
  }
  gf::Fp8Params prm = {};
  prm.M = static_cast<int32_t>(p->m);
  prm.N = static_cast<int32_t>(p->n);
  prm.groups = static_cast<int32_t>(p->groups);
  prm.num_k_blocks = static_cast<int32_t>((p->k + 127) / 128);
  prm.num_n_blocks = static_cast<int32_t>((p->n + 127) / 128);
  prm.offsets = offsets;
  prm.a_scale = a_scale;
  prm.b_scale = b_scale;
  prm.b2_scale = b2_scale;
  prm.out = out;
  prm.out_scale = out_scale;
  if (p->kernel <= kNarrow64) {
    prm.counters = static_cast<int32_t*>(p->d_work);
    prm.partials =
        reinterpret_cast<float*>(static_cast<char*>(p->d_work) + counter_bytes(p));
  }
  prm.status = p->d_status;
  prm.wait_limit_ns = p->wait_limit_ns;
  prm.drop_load = p->drop_load;

  gf::Fp8LaunchArgs la = {};
  la.tmA = &tmA;
  la.tmB = &tmB;
  la.tmB2 = dual ? &tmB2 : &tmB;
  la.params = &prm;
  la.grid = p->grid;
  la.bf16 = p->dtype == GF_BF16 ? 1 : 0;
  la.dual = dual ? 1 : 0;
  la.tile_rows = p->tile_rows;
  la.pdl = p->pdl;
  la.stream = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t err = p->kernel == kPair     ? gf::launch_fp8_wide(la)
                          : p->kernel == kSingle ? gf::launch_fp8_single(la)
                                                 : gf::launch_fp8_narrow(la);
  return err == cudaSuccess ? GF_OK : runtime_fail(GF_ERR_CUDA);
}

}  // extern "C"
