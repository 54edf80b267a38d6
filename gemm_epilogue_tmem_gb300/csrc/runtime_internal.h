// Host helpers of runtime.cu used by the library's other entry points.
#pragma once

#include <cuda.h>
#include <stddef.h>
#include <stdint.h>

#include "gf.h"

namespace gf {

// Device of the calling thread's current driver context (else the runtime's).
gf_status runtime_current_device(int* dev);

// The calling thread's current driver context (nullptr when there is none or
// the driver call is unavailable).
CUcontext runtime_current_context();

// Records `s` as the calling thread's last error (gf_last_error) and returns it.
gf_status runtime_fail(gf_status s);

// Zeroes device memory and returns once that is done. A memset on the default
// stream would still be to come when the caller goes on, and a launch on a
// non-blocking stream does not wait for it.
gf_status runtime_zero(void* ptr, size_t bytes);

// 2-D TMA map over a row-major [outer, inner] matrix of 16-bit elements with
// box_inner x box_outer boxes, 128-byte swizzle, zero fill out of bounds.
bool runtime_encode_2d(CUtensorMap* map, const void* ptr, gf_dtype dt, uint64_t inner,
                       uint64_t outer, uint32_t box_inner, uint32_t box_outer);

// The same for a row-major [outer, inner] matrix of bytes.
bool runtime_encode_2d_u8(CUtensorMap* map, const void* ptr, uint64_t inner, uint64_t outer,
                          uint32_t box_inner, uint32_t box_outer);

// A plan of an operator that is not a 16-bit GEMM (epi >= EPI_FP8) on the
// calling thread's device, checked to be one the kernels run on: defaults and
// the status word. nullptr with the reason in gf_last_error.
gf_plan* runtime_new_plan(int epi, gf_dtype dtype);

// GF_OPT_KERNEL of an e4m3 product's plan.
gf_status runtime_fp8_set_kernel(gf_plan* p, int64_t value);

// The most CTAs that share a tile of such a plan; 0 where the offsets decide.
int runtime_fp8_k_splits(const gf_plan* p);

// After a launch of such a plan that gave up: its counters back to zero.
gf_status runtime_fp8_clear_counters(gf_plan* p);

// The number of SMs of the calling thread's device, checked as above.
gf_status runtime_device(int* dev, int* sms);

}  // namespace gf
