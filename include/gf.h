/*
 * gf -- fused GEMM + epilogue on GB300 (sm_103a): the C ABI.
 *
 * One dense half-precision matrix multiply per call, with the epilogue run
 * inside the same kernel while the fp32 accumulator is still on chip:
 *
 *   out[M,N] = epilog( A[M,K] . B[K,N] )      fp16/bf16 in, fp32 accumulate
 *
 * The operations follow these web pages on fused matmul epilogs:
 *  - "Fusing Matmul Epilogs with nvmath-python": "The problem addressed by
 *    fused epilogs" (product + bias per output column + ReLU in one call),
 *    "Forward-pass capabilities in the source" (RELU_BIAS, RELU_AUX_BIAS and
 *    its bit-encoded relu_aux mask; the stateful plan / execute split),
 *    "Backward-pass path shown in the example" (DRELU_BGRAD: the product with
 *    the transposed weight, masked by relu_aux, plus the column-wise sum that
 *    is the bias gradient).
 *  - "nvmath-python 封装 cuBLASLt ..." (nvmath-python over cuBLASLt): step 1
 *    (fp16 operands, bias of shape (m,1)), step 2 (plan with
 *    COMPUTE_32F_FAST_16F: fp32 accumulation; epilog and epilog inputs fixed
 *    at plan time), step 3 (execute is asynchronous on a stream; free
 *    releases the plan), "plan reuse" (planning is the expensive step,
 *    execute is light and reused for equal shape, dtype and epilog), "other
 *    epilogs" (BIAS, GELU_BIAS).
 *
 * Conventions for every call:
 *  - Matrices are dense and row-major. A is [m, k]. B is [k, n]
 *    (GF_B_KN, the default) or given as an [n, k] matrix W with B = W^T
 *    (GF_B_NK: an nn.Linear weight, or the transposed weight of a backward
 *    pass). out is [m, n].
 *  - Device pointers are caller-owned device memory (for example torch
 *    tensors), 16-byte aligned. The library never frees them.
 *  - relu_aux words: uint32 [ceil(m/32), n] row-major. Bit (i % 32) of word
 *    [i/32][j] is 1 when the fp32 pre-activation z[i][j] = acc + bias is
 *    strictly greater than 0. Bits of rows >= m are 0.
 *  - Errors: a call that fails returns a gf_status (or NULL for the plan
 *    constructors) and records it for gf_last_error() on the calling thread.
 *    Invalid arguments are rejected before anything is enqueued.
 *  - The stream argument is a cudaStream_t (NULL: the legacy default stream),
 *    declared through its underlying struct so this header needs no CUDA
 *    header.
 */
#ifndef GF_H
#define GF_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define GF_API __attribute__((visibility("default")))
#else
#define GF_API
#endif

struct CUstream_st; /* cudaStream_t == struct CUstream_st* */

typedef enum gf_status {
  GF_OK = 0,
  GF_ERR_INVALID_VALUE = 1,   /* bad argument: NULL, size, alignment, enum  */
  GF_ERR_UNSUPPORTED = 2,     /* valid but not handled (shape rule, device) */
  GF_ERR_NO_DEVICE = 3,       /* no CUDA device could be queried            */
  GF_ERR_CUDA = 4,            /* a CUDA runtime or driver call failed       */
  GF_ERR_OUT_OF_MEMORY = 5,   /* plan workspace could not be allocated      */
  GF_ERR_DEVICE_TIMEOUT = 6   /* a bounded wait inside a kernel gave up     */
} gf_status;

typedef enum gf_dtype {
  GF_F16 = 0,  /* IEEE binary16 in and out */
  GF_BF16 = 1, /* bfloat16 in and out      */
  GF_F32 = 2  /* IEEE binary32: a router's logits only */
} gf_dtype;

typedef enum gf_epilog {
  GF_EPILOG_NONE = 0,          /* out = acc                                      */
  GF_EPILOG_RELU_BIAS = 1,     /* out = max(acc + bias, 0)                       */
  GF_EPILOG_RELU_AUX_BIAS = 2, /* RELU_BIAS, and aux_out = relu_aux words        */
  GF_EPILOG_DRELU_BGRAD = 3,   /* out = acc masked by aux_in; bgrad = colsum(out) */
  GF_EPILOG_BIAS = 4,          /* out = acc + bias                               */
  GF_EPILOG_GELU_BIAS = 5,     /* out = gelu(acc + bias), tanh form              */
  GF_EPILOG_GELU_AUX_BIAS = 6, /* GELU_BIAS, and aux_out = acc + bias (dtype)    */
  GF_EPILOG_DGELU_BGRAD = 7    /* out = acc * gelu'(aux_in); bgrad = colsum(out) */
} gf_epilog;
/* GELU is the tanh form 0.5 z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3)))
 * (Hendrycks & Gimpel 2016), named as GELU_BIAS on the nvmath-python /
 * cuBLASLt page ("other epilogs"). Its aux is the pre-activation z = acc +
 * bias rounded to dtype, [m, n] row-major: what DGELU_BGRAD reads back. */

typedef enum gf_bias_axis {
  GF_BIAS_COL = 0, /* bias[n]: one value per output column, broadcast down rows */
  GF_BIAS_ROW = 1  /* bias[m]: one value per output row (a (m,1) bias)          */
} gf_bias_axis;

typedef enum gf_b_layout {
  GF_B_KN = 0, /* B stored [k, n] row-major                        */
  GF_B_NK = 1  /* B = W^T with W stored [n, k] row-major          */
} gf_b_layout;

typedef enum gf_bgrad_mode {
  GF_BGRAD_TWO_PASS = 0, /* per-tile fp32 partial sums, then a fixed-order sum: deterministic */
  GF_BGRAD_ATOMIC = 1    /* one fp32 atomicAdd per column per tile: run-to-run order varies  */
} gf_bgrad_mode;

typedef struct gf_plan gf_plan;

/*
 * Plan one fused GEMM + epilogue: validates the problem, checks that the
 * current CUDA device is an sm_103 GPU, picks the tile configuration and
 * allocates the plan's device workspace (status word; bgrad partial sums for
 * DRELU_BGRAD). Host only; enqueues nothing. Equivalent to
 * gf_matmul_plan_ex(..., GF_B_KN).
 *
 * Source: the plan step of the stateful Matmul ("Fusing Matmul Epilogs with
 * nvmath-python", "Forward-pass capabilities in the source"; nvmath-python /
 * cuBLASLt page, step 2 and "plan reuse").
 *
 * m, n, k   : problem size, 0 <= m, n, k < 2^31; n % 8 == 0 and k % 8 == 0
 *             (16-byte row strides), else GF_ERR_UNSUPPORTED. m, n or k may be
 *             0 (an empty product; k == 0 makes acc = 0).
 * dtype     : element type of A, B, bias and out.
 * epilog    : one of gf_epilog.
 * bias_axis : GF_BIAS_COL or GF_BIAS_ROW; DRELU_BGRAD needs GF_BIAS_COL (its
 *             bias gradient is per column), else GF_ERR_UNSUPPORTED. Ignored by
 *             GF_EPILOG_NONE.
 * Returns a library-owned plan (release with gf_plan_free), or NULL with the
 * reason in gf_last_error().
 *
 * Environment overrides, read when a plan is made (gf_plan_set_option
 * called afterwards wins): GF_KERNEL (as GF_OPT_KERNEL), GF_TILE_N (128 or
 * 256, as GF_OPT_TILE_N), GF_BGRAD_MODE=atomic, GF_WAIT_LIMIT_US (as
 * GF_OPT_WAIT_LIMIT_US); GF_DEBUG prints a nonzero device status word from
 * gf_plan_status on stderr. Out-of-range values are ignored.
 */
GF_API gf_plan* gf_matmul_plan(int64_t m, int64_t n, int64_t k, gf_dtype dtype, gf_epilog epilog,
                               gf_bias_axis bias_axis);

/* gf_matmul_plan with the storage of B given explicitly (see gf_b_layout).
 * The backward of a linear layer multiplies by W^T for the forward weight W
 * ("Backward-pass path shown in the example"): that is GF_B_NK with W. */
GF_API gf_plan* gf_matmul_plan_ex(int64_t m, int64_t n, int64_t k, gf_dtype dtype,
                                  gf_epilog epilog, gf_bias_axis bias_axis,
                                  gf_b_layout b_layout);

/*
 * Enqueue the planned GEMM + epilogue on `stream` and return at once (the
 * nvmath-python / cuBLASLt page, step 3: execution does not block; the
 * caller synchronises). One kernel launch, plus one small finalize launch
 * for DRELU_BGRAD / DGELU_BGRAD in GF_BGRAD_TWO_PASS mode.
 *
 * A       : device [m, k].
 * B       : device [k, n] (GF_B_KN) or [n, k] (GF_B_NK).
 * bias    : device, n (GF_BIAS_COL) or m (GF_BIAS_ROW) elements of dtype.
 *           Required by RELU_BIAS, RELU_AUX_BIAS, BIAS, GELU_BIAS and
 *           GELU_AUX_BIAS; ignored otherwise.
 * out     : device [m, n] of dtype. Always required (when m*n > 0).
 * aux_in  : DRELU_BGRAD: relu_aux words [ceil(m/32), n] from a RELU_AUX_BIAS
 *           forward. DGELU_BGRAD: the pre-activation [m, n] of dtype from a
 *           GELU_AUX_BIAS forward. Required by both; ignored otherwise.
 * aux_out : RELU_AUX_BIAS: relu_aux words [ceil(m/32), n], written in full.
 *           GELU_AUX_BIAS: the pre-activation [m, n] of dtype. Required by
 *           both; ignored otherwise.
 * bgrad   : device fp32 [n], overwritten with the column sums of the fp32
 *           epilogue output (before rounding). Required by DRELU_BGRAD and
 *           DGELU_BGRAD; ignored otherwise.
 * A missing required pointer or a pointer not 16-byte aligned gives
 * GF_ERR_INVALID_VALUE; a failed launch gives GF_ERR_CUDA. The plan's
 * workspace is shared by its calls: use one plan from one stream at a time.
 */
GF_API gf_status gf_matmul_execute(const gf_plan* plan, const void* A, const void* B,
                                   const void* bias, void* out, const void* aux_in,
                                   void* aux_out, float* bgrad, struct CUstream_st* stream);

/*
 * Gate+up SwiGLU forward in one kernel ("gemm_swiglu_mlp_fusion.py" sample,
 * module docstring: silu(x Wg^T) * (x Wu^T) as one fused kernel, the down
 * projection a separate GEMM). Per output tile the kernel keeps two fp32
 * accumulators in tensor memory, g = x Wg^T and u = x Wu^T, and its epilogue
 * writes h = silu(g) * u with silu(g) = g / (1 + e^-g).
 *
 * m = rows of x (tokens), n = I (intermediate width), k = H (model width),
 * same size rules as gf_matmul_plan. save_gu = 1 also stores g and u
 * (rounded to dtype) for the backward ("save" rather than recompute); 0 does
 * not. The down projection out = h Wd^T is a plain
 * gf_matmul_plan_ex(m, H, I, dtype, GF_EPILOG_NONE, GF_BIAS_COL, GF_B_NK).
 */
GF_API gf_plan* gf_swiglu_plan(int64_t m, int64_t n, int64_t k, gf_dtype dtype, int save_gu);

/*
 * x: device [m, k]; Wg, Wu: device [n, k] (nn.Linear weights); h: device
 * [m, n]; g_out, u_out: device [m, n], required when the plan saves them,
 * ignored otherwise. All of dtype, 16-byte aligned. Asynchronous on stream,
 * one kernel launch. Errors as gf_matmul_execute; a plan that is not a
 * SwiGLU plan gives GF_ERR_INVALID_VALUE.
 */
GF_API gf_status gf_swiglu_execute(const gf_plan* plan, const void* x, const void* Wg,
                                   const void* Wu, void* h, void* g_out, void* u_out,
                                   struct CUstream_st* stream);

/*
 * dSwiGLU as the epilogue of dh = dout . Wd ("gemm_swiglu_mlp_fusion.py",
 * module docstring: the backward's dSwiGLU fused as the epilogue of
 * matmul(dout, Wd) -> dh). With the saved g and u:
 *   d_up   = dh * silu(g)
 *   d_gate = dh * u * sigmoid(g) * (1 + g (1 - sigmoid(g)))
 * m = rows, n = I, k = H. dout: device [m, k]; Wd: device [k, n] (the
 * down-projection weight as stored, [H, I]); g, u: device [m, n] from a
 * saving SwiGLU forward; d_gate, d_up: device [m, n]. All of dtype.
 */
GF_API gf_plan* gf_dswiglu_plan(int64_t m, int64_t n, int64_t k, gf_dtype dtype);

GF_API gf_status gf_dswiglu_execute(const gf_plan* plan, const void* dout, const void* Wd,
                                    const void* g, const void* u, void* d_gate, void* d_up,
                                    struct CUstream_st* stream);

/*
 * A product with its bias, an activation and a residual in one kernel, the last
 * step of a block that adds to a residual stream:
 *   z   = A . B + bias,   out = act(z) + residual
 * in fp32, rounded once. The activation and the residual's addition run on the
 * accumulator while it is on chip; neither z nor act(z) goes through memory (z only
 * if z_out asks for it).
 *
 * m, n, k, dtype, b_layout: as gf_matmul_plan_ex. Options: as its plans, and
 * GF_OPT_KERNEL 4, the kernel for few rows (tiles of 16, 32 or 64 rows and 128 columns; it
 * reads B once and joins the parts of a tile's k in a cluster's shared memory: no
 * workspace). It is the plan's choice up to 64 rows, and up to 128 where its tiles are
 * few. gf_matmul_autotune does not take these plans.
 */
typedef enum gf_activation {
  GF_ACT_NONE = 0, /* act(z) = z                                             */
  GF_ACT_RELU = 1, /* max(z, 0)                                              */
  GF_ACT_GELU = 2, /* GELU in its tanh form                                  */
  GF_ACT_SILU = 3  /* z / (1 + e^-z)                                         */
} gf_activation;

GF_API gf_plan* gf_matmul_residual_plan(int64_t m, int64_t n, int64_t k, gf_dtype dtype,
                                        gf_activation act, gf_b_layout b_layout);

/*
 * A, B: as gf_matmul_execute. bias: device, n elements of dtype, or NULL: none.
 * residual, out: device [m, n] of dtype; they may be the same array, which then holds
 * the sum. z_out: device [m, n] of dtype, or NULL: z is not kept (gf_dact_bgrad
 * takes it). Otherwise outputs overlap neither each other nor an input. One kernel launch,
 * asynchronous on stream; errors as gf_matmul_execute. The plan's workspace is
 * shared by its calls: one stream at a time.
 */
GF_API gf_status gf_matmul_residual_execute(const gf_plan* plan, const void* A, const void* B,
                                            const void* bias, const void* residual, void* out,
                                            void* z_out, struct CUstream_st* stream);

/*
 * The gradients of that call up to its product: with d_out the gradient of out,
 * which is the residual's as well,
 *   d_z = d_out * act'(z),   bgrad[j] = sum_i d_z[i][j]  (fp32, before rounding)
 * d_z goes on into the products of the gradients of A and B. d_z of ReLU is d_out for
 * z > 0, else 0 whatever d_out is. Sums run in an order that the plan fixes: the same bits every time.
 *
 * m, n: 0 <= m, n < 2^31, n % 8 == 0 (else GF_ERR_UNSUPPORTED). d_out, z, d_z: device
 * [m, n] of dtype; d_z may be d_out or z. bgrad: device fp32 [n], or NULL: not
 * wanted. GF_ACT_NONE: z and d_z are NULL (d_z is d_out) and bgrad is not. One launch,
 * two with bgrad; asynchronous on stream. Options: GF_OPT_PDL. The plan's workspace
 * is shared by its calls: one stream at a time.
 */
GF_API gf_plan* gf_dact_bgrad_plan(int64_t m, int64_t n, gf_dtype dtype, gf_activation act);
GF_API gf_status gf_dact_bgrad_execute(const gf_plan* plan, const void* d_out, const void* z,
                                       void* d_z, float* bgrad, struct CUstream_st* stream);

/*
 * Root-mean-square norm of rows, with the residual's addition before it, in 16
 * bits or as the e4m3 operand of gf_fp8_matmul:
 *   r = x + residual rounded to dtype (x, without a residual)
 *   y = r * weight / sqrt(mean(r^2) + eps)
 * y is of r as it is stored. Sums and y are fp32 (the sum of r^2 over a row and the products
 * r * weight have to be within its range), rounded once.
 *
 * rows >= 0, 1 <= hidden <= 32768 (more: GF_ERR_UNSUPPORTED), eps >= 0 and finite.
 * Options: GF_OPT_PDL, GF_OPT_WAIT_LIMIT_US, GF_OPT_FAULT_DROP_LOAD. gf_plan_status
 * reports a copy that never came (GF_ERR_DEVICE_TIMEOUT).
 */
GF_API gf_plan* gf_rmsnorm_plan(int64_t rows, int64_t hidden, gf_dtype dtype, float eps);

/*
 * x: device [rows, hidden] of dtype; residual: the same, or NULL: none; weight:
 * device, hidden elements of dtype. residual_out: device [rows, hidden], or NULL: r
 * is not kept (NULL without a residual, when r is x). out: y in dtype. out8 and
 * out_scale: y as gf_fp8_quantize with block_rows 1 would hold it, from the fp32 y:
 * e4m3 bytes [rows, hidden], fp32 [rows, ceil(hidden / 128)]; hidden % 16 == 0, else
 * GF_ERR_UNSUPPORTED. Either out or out8 or both; out8 and out_scale go together. The scales are those
 * of 64-bit arithmetic, also where a block's largest y lies next to the border of
 * two. residual_out and out may each be x or residual; outputs do not overlap
 * otherwise. 16-byte aligned (out_scale: 4). One launch, asynchronous on stream.
 */
GF_API gf_status gf_rmsnorm_execute(const gf_plan* plan, const void* x, const void* residual,
                                    const void* weight, void* residual_out, void* out, void* out8,
                                    float* out_scale, struct CUstream_st* stream);

/*
 * Its gradients, from the gradient d_out of y and, along the residual stream,
 * d_residual of r (NULL: none). With h = r / sqrt(mean(r^2) + eps) and g = d_out * weight:
 *   d_x = (g - h mean(g h)) / sqrt(mean(r^2) + eps) + d_residual
 *   d_weight = sum over the rows of d_out * h
 * d_x is the gradient of x and of the residual alike. r: residual_out of the
 * forward (x, without a residual); nothing else of the forward is needed. d_x: device [rows,
 * hidden] of dtype, may be d_out or d_residual. d_weight: device fp32 [hidden], or NULL: not
 * wanted; its sums run in an order that the plan fixes. One launch, two with d_weight;
 * asynchronous on stream. The plan's workspace, the partial sums of d_weight, is allocated by
 * the first call that wants them (GF_ERR_OUT_OF_MEMORY; that call may be captured into a
 * graph) and shared by its calls: one stream at a time.
 */
GF_API gf_status gf_rmsnorm_grad_execute(const gf_plan* plan, const void* d_out, const void* r,
                                         const void* weight, const void* d_residual, void* d_x,
                                         float* d_weight, struct CUstream_st* stream);

/*
 * A router's choice: each token's experts and their weights, from its logits l.
 *   s = softmax(l), or 1 / (1 + e^-l) for each expert (gf_score), over the experts
 *   c = s + bias; without a bias experts are compared by l, which has their order
 * An expert is left out where l or c is -inf. With groups > 1 the experts are in `groups`
 * groups of as many consecutive ones, and only those of the topk_groups best groups
 * are chosen from: a group's score is its best c (group_best 1) or the sum of its two
 * best (2; of s without a bias; of one where it has no second). Then
 *   expert[t][0 .. topk - 1] = the experts of the largest c, the largest first
 *   weight[t][j] = scale * s[expert[t][j]], renorm: over the sum of the token's chosen s
 * Of equal ones the lowest index goes first, experts and groups. Slots that find no
 * expert left get -1 and weight 0 (gf_moe_dispatch drops them). NaN ranks above every
 * number, and is in the weights what the formulas make of it. Scores that fp32 does not tell
 * apart are compared in 64 bits. Renormalised weights are the ratios of the scores, also
 * where fp32 does not hold these; chosen scores that sum to 0 in 64 bits (logits of less than
 * -745, under softmax below the largest) have the weights 0 and pass no gradient. Else
 * logits and scores are fp32 whatever dtype is.
 *
 * tokens >= 0, 1 <= experts <= 1024, 1 <= topk <= 64, tokens * topk < 2^31, topk at most the
 * experts of topk_groups groups, groups a divisor of experts, else GF_ERR_INVALID_VALUE; at most 32
 * groups, else GF_ERR_UNSUPPORTED. dtype: of the logits, GF_F32 too. ld: elements
 * between the rows of logits and of d_logits, experts <= ld <= 2^24 (a router's product
 * may have more columns than there are experts). Options: GF_OPT_PDL; no workspace.
 */
typedef enum gf_score { GF_SCORE_SOFTMAX = 0, GF_SCORE_SIGMOID = 1 } gf_score;

GF_API gf_plan* gf_route_plan(int64_t tokens, int64_t experts, int64_t topk, gf_dtype dtype,
                              gf_score score, int32_t renorm, float scale, int64_t groups,
                              int64_t topk_groups, int32_t group_best, int64_t ld);

/*
 * logits: device [tokens, ld] of dtype, of which the first `experts` columns are
 * read; bias: device fp32 [experts], or NULL: none. expert: device int32 [tokens,
 * topk] and weight: device fp32 [tokens, topk], what gf_moe_dispatch and gf_moe_combine
 * take. 16-byte aligned (bias: 4). One launch, asynchronous on stream.
 */
GF_API gf_status gf_route_execute(const gf_plan* plan, const void* logits, const float* bias,
                                  int32_t* expert, float* weight, struct CUstream_st* stream);

/*
 * The gradient of the logits from that of the weights, the choice held (the bias
 * takes part in the choice alone). expert: of the forward; entries outside [0,
 * experts) have no part, and the d_weight beside them is not used. d_weight: device fp32
 * [tokens, topk] (of gf_moe_combine_grad); d_logits: device [tokens, ld] of dtype, columns from
 * `experts` on set to 0. One launch, asynchronous on stream.
 */
GF_API gf_status gf_route_grad_execute(const gf_plan* plan, const void* logits,
                                       const int32_t* expert, const float* d_weight,
                                       void* d_logits, struct CUstream_st* stream);

/*
 * Mixture-of-experts routing: the rows of a token batch, sorted by expert and
 * back.
 *
 * A router gives each of `tokens` tokens `topk` experts, expert[t][s], and
 * weights, weight[t][s]. Slot i = t * topk + s is kept when 0 <= expert < experts,
 * and dropped otherwise (-1: past an expert's capacity). The kept slots,
 * ordered by expert and within one expert by i (a stable sort), are the rows:
 *   offsets[e]  = the first row of expert e; offsets[experts] = kept slots
 *   row_of[t][s] = the slot's row, -1 when dropped
 *   slot_of[r]  = the slot of row r, -1 for rows >= offsets[experts]
 *   dispatch      rows[row_of[t][s]] = x[t]            (rows without a slot: 0)
 *   its gradient  d_x[t] = sum_s d_rows[row_of[t][s]]
 *   combine       out[t] = sum_s weight[t][s] rows[row_of[t][s]]
 *   its gradient  d_rows[row_of[t][s]] = weight[t][s] d_out[t]  (without a slot: 0)
 *                 d_weight[t][s] = <d_out[t], rows[row_of[t][s]]>  (dropped: 0)
 * Sums run in fp32 in slot order, so results do not vary from run to run. A
 * token whose slots are all dropped gets zeros.
 *
 * tokens >= 0, 1 <= topk <= 64, 1 <= experts <= 1024, 1 <= hidden <= 2^24,
 * tokens * topk < 2^31. The calls need no workspace. GF_OPT_PDL is the plan's
 * one option; gf_plan_status, gf_plan_describe (tile_m: tokens per CTA of the
 * sort), gf_plan_launches (of gf_moe_dispatch_execute) and gf_plan_free take
 * it as any other plan.
 */
GF_API gf_plan* gf_moe_plan(int64_t tokens, int64_t topk, int64_t experts, int64_t hidden,
                            gf_dtype dtype);

/*
 * Sort and copy. expert: device int32 [tokens, topk]; x: device [tokens,
 * hidden] of dtype; offsets: device int32 [experts + 1]; row_of: device int32
 * [tokens, topk]; slot_of: device int32 [tokens * topk]; rows: device [tokens *
 * topk, hidden] of dtype. x and rows may both be NULL: the sort alone. Arrays
 * must not overlap. Asynchronous on stream; pointers 16-byte aligned
 * (GF_ERR_INVALID_VALUE otherwise, as for a plan of another kind). So for the
 * three calls below.
 */
GF_API gf_status gf_moe_dispatch_execute(const gf_plan* plan, const int32_t* expert, const void* x,
                                         int32_t* offsets, int32_t* row_of, int32_t* slot_of,
                                         void* rows, struct CUstream_st* stream);

/* gf_moe_dispatch_execute whose rows are quantised on the way, each token once,
 * as gf_fp8_quantize with block_rows 1 would: rows: device e4m3 bytes [tokens *
 * topk, hidden], scale: device fp32 [tokens * topk, ceil(hidden / 128)] (rows
 * without a slot: zeros with scale 1). hidden % 16 == 0, else
 * GF_ERR_UNSUPPORTED. All pointers required. */
GF_API gf_status gf_moe_dispatch_fp8_execute(const gf_plan* plan, const int32_t* expert,
                                             const void* x, int32_t* offsets, int32_t* row_of,
                                             int32_t* slot_of, void* rows, float* scale,
                                             struct CUstream_st* stream);

/* The gradient of dispatch: d_x: device [tokens, hidden], d_rows: device
 * [tokens * topk, hidden], both of dtype. An entry of row_of outside [0, tokens *
 * topk) counts as dropped, here and in the two calls below. */
GF_API gf_status gf_moe_dispatch_grad_execute(const gf_plan* plan, const int32_t* row_of,
                                              const void* d_rows, void* d_x,
                                              struct CUstream_st* stream);

/* Back to the tokens, weighted: weight: device fp32 [tokens, topk]; rows: device
 * [tokens * topk, hidden] and out: device [tokens, hidden], both of dtype. The
 * weight of a dropped slot is not used (it may be NaN). */
GF_API gf_status gf_moe_combine_execute(const gf_plan* plan, const int32_t* row_of,
                                        const float* weight, const void* rows, void* out,
                                        struct CUstream_st* stream);

/* The gradient of combine: offsets (its last entry bounds the rows that hold a
 * slot), row_of, weight and rows as in the forward, d_out: device [tokens,
 * hidden]; d_rows: device [tokens * topk, hidden] of dtype, d_weight: device
 * fp32 [tokens, topk], both written in full. */
GF_API gf_status gf_moe_combine_grad_execute(const gf_plan* plan, const int32_t* offsets,
                                             const int32_t* row_of, const float* weight,
                                             const void* rows, const void* d_out, void* d_rows,
                                             float* d_weight, struct CUstream_st* stream);

/*
 * 8-bit floating point with a scale for each block of 128: x is held as e4m3
 * values q (OCP 8-bit floating point: 4 exponent bits, 3 mantissa bits, largest
 * 448, no infinity) times one fp32 scale per block of block_rows x 128
 * elements, block_rows 1 (activations) or 128 (weights).
 *   scale = the smallest power of two with max|x| / scale <= 448 over the
 *           block's finite elements, at least 2^-126; 1 for a block without a
 *           finite non-zero element
 *   q     = x / scale rounded to nearest even; infinities and NaN become NaN
 * A power of two makes the division exact, so the rounding to e4m3 is the only
 * one; it costs at most one bit of e4m3's exponent range. x: device [m, k] of
 * dtype; q: device bytes [m, k]; scale: device fp32 [ceil(m / block_rows),
 * ceil(k / 128)]. 0 <= m, k < 2^31, k % 16 == 0 (else GF_ERR_UNSUPPORTED).
 * x and q 16-byte aligned; scales, here and below, as fp32 values are (4 bytes),
 * so that a part of a larger array will do.
 * Asynchronous on stream; needs no plan and no workspace.
 */
GF_API gf_status gf_fp8_quantize(int64_t m, int64_t k, gf_dtype dtype, int32_t block_rows,
                                 const void* x, void* q, float* scale,
                                 struct CUstream_st* stream);

typedef enum gf_fp8_epilog {
  GF_FP8_EPILOG_NONE = 0,         /* out = the product, of dtype                           */
  GF_FP8_EPILOG_SWIGLU_QUANT = 1  /* out = e4m3 of silu(gate) * up, out_scale its scales    */
} gf_fp8_epilog;

/*
 * Plan out = A . B^T with e4m3 operands and a scale for each block of 128,
 * over `groups` groups of rows that each have a B of their own (the experts):
 *   out[i][j] = sum_b a_scale[i][b] b_scale[g][j / 128][b]
 *                     sum_{l in block b} A[i][l] B[g][j][l]      b = l / 128
 * with g the group of row i. Each block's sum of up to 128 products and the
 * sum over the blocks are fp32. GF_FP8_EPILOG_SWIGLU_QUANT forms two products,
 * gate = A . B^T and up = A . B2^T, and writes h = silu(gate) * up quantised
 * as by gf_fp8_quantize with block_rows 1 from the fp32 h: the next product's A.
 *
 * m rows, n columns, k; groups >= 1. 0 <= m, n, k < 2^31, 1 <= groups <= 1024.
 * k % 16 == 0 (16-byte rows for the tensor maps), n % 8 == 0, or n % 16 == 0
 * for SWIGLU_QUANT, and m, groups * n up to 2^31 - 513, at most 2^30 tiles of 16 x
 * 128, else GF_ERR_UNSUPPORTED. dtype: the element type of out
 * (NONE). Options: GF_OPT_KERNEL (0 the plan's choice, the one that takes the least
 * time by a model of the four for groups of about alike numbers of rows; 1 and 2
 * the kernel for few rows with tiles of 16 and 64 rows; 3 the single-CTA kernel
 * with tiles of 128; 4 the CTA-pair kernel with tiles of 256), GF_OPT_PDL, GF_OPT_WAIT_LIMIT_US,
 * GF_OPT_FAULT_DROP_LOAD; others give GF_ERR_UNSUPPORTED.
 */
GF_API gf_plan* gf_fp8_matmul_plan(int64_t m, int64_t n, int64_t k, int64_t groups,
                                   gf_dtype dtype, gf_fp8_epilog epilog);

/*
 * A: device e4m3 [m, k]; a_scale: device fp32 [m, ceil(k / 128)]. B, B2: device
 * e4m3 [groups, n, k]; b_scale, b2_scale: device fp32 [groups, ceil(n / 128),
 * ceil(k / 128)]; B2 and b2_scale: SWIGLU_QUANT only. Scales are any fp32 values;
 * some kernels form a_scale * b_scale first, so that a product of the two which
 * overflows fp32 or falls below 2^-126 gives what fp32 makes of it.
 * offsets: device int32 [groups + 1], group g is rows offsets[g] ..
 * offsets[g + 1] - 1 (offsets[0] is taken as 0 and each other one bounded to
 * [the one before, m] by the kernel); NULL with groups == 1: all rows. Rows of
 * no group get zeros (and scale 1).
 * out: device [m, n] of dtype (NONE), or e4m3 bytes [m, n] with out_scale:
 * device fp32 [m, ceil(n / 128)] (SWIGLU_QUANT). 16-byte aligned;
 * asynchronous on stream, one kernel launch; the host never reads offsets.
 * The plan's workspace is shared by its calls: one stream at a time.
 */
GF_API gf_status gf_fp8_matmul_execute(const gf_plan* plan, const void* A, const float* a_scale,
                                       const void* B, const float* b_scale, const void* B2,
                                       const float* b2_scale, const int32_t* offsets, void* out,
                                       float* out_scale, struct CUstream_st* stream);

/*
 * Synchronise `stream`, then read and clear the plan's device status word.
 * Returns GF_ERR_DEVICE_TIMEOUT if a bounded wait in a kernel of this plan
 * gave up since the last call (the kernel then skipped the rest of its work
 * and returned; its outputs are incomplete), GF_ERR_CUDA if the stream
 * reports an error, else GF_OK. Not on the pages: the library's failure
 * detection.
 */
GF_API gf_status gf_plan_status(const gf_plan* plan, struct CUstream_st* stream);

/*
 * Plan options (not on the pages; tuning and failure-detection knobs).
 * GF_OPT_BGRAD_MODE      : a gf_bgrad_mode (default GF_BGRAD_TWO_PASS).
 * GF_OPT_WAIT_LIMIT_US   : the limit of every bounded wait inside the kernel,
 *                          in microseconds (default 2000000, min 1000).
 * GF_OPT_TILE_N          : output tile width, 128 or 256 (0: the plan's choice).
 * GF_OPT_FAULT_DROP_LOAD : test hook. When v > 0 the producer skips its v-th
 *                          stage load, so the consumer's bounded wait runs
 *                          out; execute then completes with
 *                          GF_ERR_DEVICE_TIMEOUT from gf_plan_status. 0: off.
 * GF_OPT_KERNEL          : 0 the plan's choice (the CTA-pair kernel when its
 *                          256-row tiles fill the resident pairs, with
 *                          256 x 512 tiles when k >= 2048 and their
 *                          schedule -- waves of the resident pairs, with the
 *                          last-wave split of GF_OPT_SPLIT_K -- is no longer
 *                          than the 256 x 256 tiles' weighed by the wide
 *                          tile's gain, 12 % (4 % for the gate+up SwiGLU
 *                          plans); else the single-CTA kernel),
 *                          1 the single-CTA kernel
 *                          (128 x tile_n tiles), 2 the CTA-pair kernel
 *                          (256 x 256 tiles on two SMs, 256 x 128 for the
 *                          gate+up SwiGLU plans; GF_ERR_UNSUPPORTED if it
 *                          cannot be resident on this device), 3 the
 *                          CTA-pair kernel with 256 x 512 tiles (256 x 256
 *                          for the gate+up SwiGLU plans, each output column
 *                          taking a column of both weights: 3/4 of the
 *                          operand traffic per flop, one accumulator whose
 *                          halves are released as soon as the epilogue has
 *                          them in registers). Plans of
 *                          gf_matmul_residual_plan: 4 the kernel for few
 *                          rows, which of the options below takes
 *                          GF_OPT_SPLIT_K and GF_OPT_PDL alone.
 * Returns GF_ERR_INVALID_VALUE for an unknown option or value.
 */
typedef enum gf_option {
  GF_OPT_BGRAD_MODE = 0,
  GF_OPT_WAIT_LIMIT_US = 1,
  GF_OPT_TILE_N = 2,
  GF_OPT_FAULT_DROP_LOAD = 3,
  GF_OPT_KERNEL = 4,
  GF_OPT_GROUP_M = 5,
  GF_OPT_L2_HINTS = 6,
  GF_OPT_SCHEDULE = 7,
  GF_OPT_SPLIT_K = 8,
  GF_OPT_PDL = 9,
  GF_OPT_RASTER = 10
} gf_option;
/* GF_OPT_SCHEDULE: how persistent CTAs (or CTA pairs) walk the output tiles,
 * overlapping each tile's epilogue with the next tile's mainloop.
 *   0 the plan's choice: 2 for the CTA-pair kernel, 3 for the single-CTA one;
 *   1 one tile per CTA (pair), launched in raster order by the hardware;
 *   2 dynamic (CTA-pair kernel): each pair takes the next tile from a counter
 *     in the plan's workspace, so the tiles in flight stay a contiguous run of
 *     the raster order and share their operand panels in L2;
 *   3 static: pair (CTA) c takes tiles c, c + grid, c + 2 grid, ... */
/* GF_OPT_L2_HINTS: L2 eviction priority of the operand loads, 10 * a + b with
 * a (for A) and b (for B) each 0 = no hint, 1 = evict first (streamed),
 * 2 = evict last (re-read by the tiles that follow). */
/* GF_OPT_GROUP_M: output tiles are visited in groups of this many row blocks
 * (128 rows, or 256 for the CTA-pair kernel) -- or column blocks, see
 * GF_OPT_RASTER -- so that concurrently running tiles share operand panels
 * in L2. 0: the plan's choice (8, or 4 column blocks for the 256 x 512
 * tiles); 1..4096 otherwise. */
/* GF_OPT_SPLIT_K: the single-CTA kernel shares the k-blocks of each output
 * tile among this many CTAs (one B operand only); so does the CTA-pair kernel
 * with 256 x 256 or 256 x 512 tiles for GF_EPILOG_NONE plans (each of its
 * CTAs then has a partial sum and a counter of its own, and the last to
 * finish for its 128 rows adds them; the plan's choice there splits only the
 * tiles of a last wave that is at most half full, when k has at least 32
 * blocks, or 128 when the tiles fill more than three waves, and it takes the
 * 256 x 512 tiles when their split schedule is the shorter one).
 * Each CTA leaves its fp32 partial sum in the plan's workspace; the last one
 * of a tile to finish adds the partials in split order (the result does not
 * depend on which finishes last) and runs the epilogue, so no CTA waits for
 * another. 0: the plan's choice (a split when k has at least 16 blocks of 64
 * and the tiles fill at most half the SMs: as many splits as the idle SMs
 * take, at most 8 and at most sqrt(k / 128)); 1: no split; 2..64: that many
 * (fewer when k has fewer 64-wide blocks; none when the partial sums would
 * take more than 256 MB). The workspace grows to tiles x splits x 128 x tile_n
 * fp32 plus one counter per tile; GF_ERR_OUT_OF_MEMORY (and no split) when it
 * cannot be allocated. Set options only while no launch of the plan is in
 * flight. Plans of gf_matmul_residual_plan split as GF_EPILOG_NONE plans do; their kernel
 * for few rows shares a tile among a cluster of up to 8 CTAs, by default as many as
 * can be resident for all tiles at once. */
/* GF_OPT_RASTER: the order of the output tiles. 1: raster groups of
 * GF_OPT_GROUP_M row blocks, column by column within a group (the group's
 * A panels stay in L2 while B streams through); 2: groups of GF_OPT_GROUP_M
 * column blocks, row by row within a group (B panels stay in L2); 0 (default)
 * the plan's choice: 2 with groups of 4 for the 256 x 512 tiles, else 1 with
 * groups of 8. Results are the same in every order. */
/* GF_OPT_PDL: 1 (default) launches the plan's kernels as programmatic
 * dependent launches: a kernel's launch and set-up (barriers, tensor memory,
 * descriptor prefetch) overlap the end of the kernel before it on the stream,
 * and it touches global memory only once that kernel has completed and its
 * writes are visible, so results are the same as with 0 (plain stream
 * order). */

GF_API gf_status gf_plan_set_option(gf_plan* plan, gf_option option, int64_t value);

/*
 * Plan-time autotuning of a gf_matmul plan (the plan-time algorithm search of
 * the nvmath-python / cuBLASLt page, "limitations" paragraph: autotuning
 * through MatmulPlanPreferences; here a search over this library's own
 * kernels). Runs the planned product once per candidate (CTA-pair kernel
 * with 256- or 512-wide tiles, dynamic or static schedule and raster groups
 * of 4, 8 or 16 tile rows; single-CTA kernel with 256- or 128-wide tiles,
 * and with 128-wide tiles k split 1, 2, 4 or 8 ways) on the caller's buffers,
 * `reps` timed launches each after one warm-up, synchronising `stream`, and
 * keeps the fastest in the plan. The outputs hold the result of the last
 * launch. Arguments as gf_matmul_execute; reps in 1..100.
 */
GF_API gf_status gf_matmul_autotune(gf_plan* plan, const void* A, const void* B,
                                    const void* bias, void* out, const void* aux_in,
                                    void* aux_out, float* bgrad, struct CUstream_st* stream,
                                    int32_t reps);

/* Read back the plan's choices: tile_m, tile_n, stages, grid size (CTAs per
 * launch), workspace bytes. Any out-pointer may be NULL. Of gf_route_plan: the call without
 * a bias, tile_m the tokens of a CTA at a time. Of gf_rmsnorm_plan: the norm in 16 bits
 * without a residual, tile_m the rows of a CTA at a time, stages those of the ring that its
 * rows come through (0: none). Of gf_dact_bgrad_plan: the first launch, tile_m the rows of
 * a CTA. */
GF_API gf_status gf_plan_describe(const gf_plan* plan, int32_t* tile_m, int32_t* tile_n,
                                  int32_t* stages, int32_t* grid, int64_t* workspace_bytes);

/* The number of CTAs that share the k-blocks of one output tile in the
 * plan's current configuration (1: no split). For an e4m3 product of one group
 * the most for any tile, with all m rows the group's; 0 for several groups on the
 * kernel for few rows, whose offsets decide it on the device.
 * GF_ERR_INVALID_VALUE for a NULL argument. */
GF_API gf_status gf_plan_k_splits(const gf_plan* plan, int32_t* k_splits);

/* The number of kernels one execute of the plan enqueues in its current
 * configuration: 0 for an empty output, else 1, plus 1 for the bias-gradient
 * epilogs in GF_BGRAD_TWO_PASS mode (the finalize kernel that adds the
 * partials; GF_BGRAD_ATOMIC enqueues a memset of bgrad instead). For a plan of
 * gf_route_plan or gf_rmsnorm_plan 1 (a gradient of the norm's weight adds one), of
 * gf_dact_bgrad_plan 2 (without bgrad 1).
 * GF_ERR_INVALID_VALUE for a NULL argument. */
GF_API gf_status gf_plan_launches(const gf_plan* plan, int32_t* launches);

/*
 * DRELU_BGRAD that allocates nothing. The pages have no counterpart: this
 * entry point exists for callers that cannot call cudaMalloc (or any
 * allocating routine) -- code that must only use memory handed to it, such
 * as a framework's memory pool, a real-time loop that must not enter the
 * allocator, or a host API that forbids allocation while it runs. A plan
 * (gf_matmul_plan_ex) allocates its workspace; this call does not.
 *
 * It computes exactly what gf_matmul_execute computes for a
 * GF_EPILOG_DRELU_BGRAD plan in GF_BGRAD_TWO_PASS mode (same kernels, same
 * arguments: A, B, out, aux_in, bgrad as documented there) and returns at
 * once after enqueuing on `stream`.
 *
 * Scratch: the per-128-row-block partial sums live in one fixed device array
 * inside the library, GF_NOALLOC_MAX_PARTIALS fp32 values (8 MiB) plus a
 * 256-byte status word. Every GPU that loads the library holds it until the
 * process exits. ceil(m/128) * n must not exceed GF_NOALLOC_MAX_PARTIALS
 * (else GF_ERR_UNSUPPORTED, nothing enqueued).
 *
 * The first call on a device (and the first after its context was torn down
 * and re-created, e.g. by a device reset) looks up the array's device
 * address for that device (cudaGetSymbolAddress; no allocation); make that
 * first call before any stream capture. Every call shares the one array and
 * reuses it as the previous call left it: each call clears the status word on
 * its stream before its kernel starts, and every partial sum the finalize
 * reads is written by that call's kernel; calls that overlap on the GPU
 * (other streams, other threads) race on it and must be serialised by the
 * caller. A bounded wait that gives up inside the kernel is recorded in the
 * array's status word; gf_noalloc_status reports it.
 *
 * Returns GF_OK, GF_ERR_INVALID_VALUE (bad size, enum, NULL or misaligned
 * pointer), GF_ERR_UNSUPPORTED (n or k not a multiple of 8, beyond the
 * scratch limit, not an sm_103 device), GF_ERR_NO_DEVICE or GF_ERR_CUDA.
 */
#define GF_NOALLOC_MAX_PARTIALS 2097152

GF_API gf_status gf_drelu_bgrad_noalloc(int64_t m, int64_t n, int64_t k, gf_dtype dtype,
                                        gf_b_layout b_layout, const void* A, const void* B,
                                        void* out, const void* aux_in, float* bgrad,
                                        struct CUstream_st* stream);

/*
 * The status of gf_drelu_bgrad_noalloc on the calling thread's current
 * device, the counterpart of gf_plan_status for that allocation-free call
 * (it allocates nothing either). Synchronises `stream`, then reads the
 * status word of the library's fixed scratch array: GF_ERR_DEVICE_TIMEOUT
 * (and the word is cleared) if a bounded wait in the most recent call's
 * kernel gave up, whose outputs are then incomplete; GF_ERR_CUDA if the
 * stream reports an error; else GF_OK. GF_ERR_NO_DEVICE / GF_ERR_UNSUPPORTED
 * as gf_drelu_bgrad_noalloc. The pages have no counterpart.
 */
GF_API gf_status gf_noalloc_status(struct CUstream_st* stream);

/* Release the plan and its workspace ("free" on the nvmath-python / cuBLASLt
 * page, step 3). Caller tensors are untouched. NULL is a no-op. Work already
 * enqueued with the plan must have completed. */
GF_API void gf_plan_free(gf_plan* plan);

/* Static text for a status code. */
GF_API const char* gf_status_string(gf_status status);

/* The status of the last failing call on this thread (GF_OK if none). */
GF_API gf_status gf_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* GF_H */
