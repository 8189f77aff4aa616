/*
 * moe_fp8.h -- C ABI of the FP8 operators beside the quantized routed
 * mixture-of-experts layer (include/moe.h), for AMD Instinct MI355X (gfx950).
 *
 * The pages' native package keeps the routed experts in FP4 and the model in
 * its original FP8/FP4 format (Anemll/ds4-ssd README, section "Run SSD
 * Sidecar Mode"; the 10100.com article on ds4-ssd, original-format package).
 * These entry points take matrices of that FP8 form:
 *
 *   tokens   a  [rows][K]: E4M3 codes (OCP, no infinities; 0x7F and 0xFF are
 *            NaN) and fp32 scales [rows][ceil(K/128)], one per run of 128
 *            consecutive values of a row;
 *   weights  w  [N][K]: E4M3 codes and fp32 scales
 *            [ceil(N/128)][ceil(K/128)], one per block of 128 x 128.
 *
 * A value is its code times its scale; the runs and blocks at the end of an
 * axis may be shorter.  With S = ceil(K/128) steps, a product is
 *
 *   out[m][n] = sum_{s<S} a_scale[m][s] * w_scale[n/128][s] *
 *               sum_{k in step s} a[m][k] * w[n][k]
 *
 * The chain of a serving step: moe_add_rmsnorm (residual stream -> bf16 rows
 * for the router and E4M3 rows for the experts), moe_route_topk and
 * moe_dispatch (include/moe.h), moe_expert_gate_up_fp8, moe_grouped_gemm_fp8
 * (down) and moe_combine; moe_layer_fp8 runs all but the first in one call.
 * moe_gemm_fp8 is the dense product of the projections around the layer.
 *
 * Conventions as in include/moe.h: device pointers, caller-owned buffers, no
 * allocation, every call only enqueues on `stream` (a stream of the current
 * device), host-side validation before any HIP call, negative status codes
 * (enum moe_status).  Calls are independent: nothing is kept between them.
 * Every call may be captured into a HIP graph.  Results do not depend on
 * timing: no floating-point atomics, sums in a fixed order.
 *
 * Alignment: codes, x, residual, weight, y, out, act and ws 16 bytes; scales
 * and int32 arrays 4 bytes.  Inputs and outputs must not overlap except
 * where stated.
 */
#ifndef QUANTIZED_ROUTED_MOE_AMD_MOE_FP8_H
#define QUANTIZED_ROUTED_MOE_AMD_MOE_FP8_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Value types of the arguments that come in more than one. */
enum moe_type {
    MOE_TYPE_BF16 = 1,
    MOE_TYPE_F32 = 2
};

/* Residual addition and root-mean-square norm of T rows of d values, with an
   optional output in E4M3:

     h = x[t] + residual[t], rounded to the residual's type and stored to
         residual_out[t] (without a residual: h = x[t])
     v = h * (1 / sqrt(mean(h^2) + eps)) * weight          (fp32)
     y[t] = bf16(v)
     q_scales[t][b] = max(max|v| / 448, 2^-126) over run b of 128
     q[t] = E4M3(v / q_scales[t][b])                        (nearest even)

   The norm reads the stored h, so it can be recomputed from the stream.
   The mean and v are fp32.  Non-finite v: a NaN becomes the code NaN and
   does not enter its run's maximum; a run holding an infinity has scale
   +inf and NaN codes at its infinities.

   x, residual, residual_out: x_type / residual_type (MOE_TYPE_BF16 or
   MOE_TYPE_F32), rows x_stride, residual_stride, residual_out_stride
   VALUES apart (each a multiple of 16 bytes; those of outputs >= d; an
   input's may be 0, one row for all).  residual and residual_out are both
   NULL or both given; residual_out may be residual itself (in place, same
   stride).  weight: weight_type [d] or NULL (1).  y: bf16 [T][d] or NULL.
   q, q_scales: E4M3 [T][d] and fp32 [T][ceil(d/128)], both or neither; at
   least one of y, q and residual_out must be given.
   Limits: T >= 0, d a positive multiple of 32 up to 2^20, eps finite and
   >= 0.  Errors: MOE_ERR_NULL, MOE_ERR_SHAPE (limits, strides),
   MOE_ERR_FORMAT (unknown type), MOE_ERR_ALIGN, MOE_ERR_UNSUPPORTED
   (residual_out overlapping residual with another stride), MOE_ERR_HIP. */
int moe_add_rmsnorm(int32_t T, int32_t d, const void* x, int32_t x_type, int64_t x_stride, const void* residual,
                    void* residual_out, int32_t residual_type, int64_t residual_stride, int64_t residual_out_stride,
                    const void* weight, int32_t weight_type, float eps, uint16_t* y, uint8_t* q, float* q_scales,
                    hipStream_t stream);

/* Dense product out [M][N] = a [M][K] . w [N][K]^T of the form above.
   a's rows lie a_stride bytes apart (a multiple of 16, >= K); out's lie
   out_stride values apart (>= N) and are MOE_TYPE_BF16 or MOE_TYPE_F32.
   Results accumulate exact products of the codes (as bf16 operands) in fp32,
   whatever the size of the call; a bf16 result is that sum rounded once.
   Limits: M >= 0 (0 enqueues nothing), N >= 1, both below 2^30; K a positive
   multiple of 32 up to 2^22; the workgroups, one per tile of 128 rows x 256
   columns and some that make the rounds over eight XCDs whole, fewer than 2^23
   (fewer than 2^22 tiles always fit).  Errors: MOE_ERR_NULL, MOE_ERR_SHAPE,
   MOE_ERR_FORMAT, MOE_ERR_ALIGN, MOE_ERR_HIP. */
int moe_gemm_fp8(int32_t M, int32_t N, int32_t K, const uint8_t* a, int64_t a_stride, const float* a_scales,
                 const uint8_t* w, const float* w_scales, void* out, int32_t out_type, int64_t out_stride,
                 hipStream_t stream);

/* The product grouped by expert: sorted row r of expert e, that is
   offsets[e] <= r < offsets[e+1] (moe_dispatch), is

     out[r] = a[src(r)] . w[e]^T,   src(r) = perm ? perm[r] / k : r

   R sorted rows, E experts; a: [a_rows][K], w: E4M3 [E][N][K] with scales
   [E][ceil(N/128)][ceil(K/128)]; offsets int32 [E+1]; perm int32 [R] or NULL
   (then a_rows >= R); out [R][N], MOE_TYPE_F32 or MOE_TYPE_BF16, precision
   as moe_gemm_fp8.  Rows of no expert (from offsets[E] on, and below
   offsets[0] where that is not 0) are written as zeros.  Experts without rows
   are not read.  Offsets outside [0, R] and rows src(r) outside [0, a_rows) are
   clamped into range, never followed.
   Limits: R >= 0 (0 enqueues nothing), 1 <= E <= 64, N and K as
   moe_gemm_fp8, k >= 1, a_rows >= 1, workgroups as there with at most
   (R + 127 min(E + 2, R)) / 128 runs of rows.  Errors as moe_gemm_fp8. */
int moe_grouped_gemm_fp8(int32_t R, int32_t E, int32_t N, int32_t K, const uint8_t* a, int32_t a_rows,
                         const float* a_scales, const uint8_t* w, const float* w_scales, const int32_t* offsets,
                         const int32_t* perm, int32_t k, void* out, int32_t out_type, hipStream_t stream);

/* Gate/up projections with SwiGLU, the result in E4M3: for sorted row r of
   expert e (token perm[r] / k of a [T][d])

     v = silu(gate[e] . a) * (up[e] . a)                    (fp32)
     act_scales[r][b] = max(max|v| / 448, 2^-126) over run b of 128
     act[r] = E4M3(v / act_scales[r][b])

   which is the `a` of a moe_grouped_gemm_fp8 with the down matrices (perm
   NULL).  gate, up: E4M3 [E][f][d] with scales [E][ceil(f/128)][ceil(d/128)];
   act E4M3 [T*k][f], act_scales fp32 [T*k][ceil(f/128)]; non-finite v as
   moe_add_rmsnorm.  Rows of no expert are left as they were.
   ws: moe_expert_gate_up_fp8_workspace_bytes(shape) bytes (0: ws may be
   NULL), uninitialised; one call at a time.  Limits as include/moe.h
   (moe_shape) with d <= 2^22 (and f, in moe_layer_fp8), workgroups as above
   with tiles of 128 columns and E for E + 2; offsets and perm clamped as above.
   Errors as moe_expert_ffn. */
size_t moe_expert_gate_up_fp8_workspace_bytes(const moe_shape* shape);
int moe_expert_gate_up_fp8(const moe_shape* shape, const uint8_t* a, const float* a_scales, const uint8_t* gate,
                           const float* gate_scales, const uint8_t* up, const float* up_scales,
                           const int32_t* offsets, const int32_t* perm, uint8_t* act, float* act_scales, void* ws,
                           size_t ws_bytes, hipStream_t stream);

/* The experts of one FP8 layer: gate and up [E][f][d], down [E][d][f]. */
typedef struct moe_fp8_experts {
    const uint8_t* gate;
    const float* gate_scales;
    const uint8_t* up;
    const float* up_scales;
    const uint8_t* down;
    const float* down_scales;
} moe_fp8_experts;

/* The layer of include/moe.h with FP8 experts: moe_route_topk on x,
   moe_dispatch, moe_expert_gate_up_fp8 on (xq, xq_scales), the down
   moe_grouped_gemm_fp8 (fp32) and moe_combine, bit for bit the calls in
   sequence.  x bf16 [T][d] and its E4M3 form xq [T][d], xq_scales
   [T][ceil(d/128)] are two outputs of one moe_add_rmsnorm (x may be NULL
   where w_router is).  Other arguments as moe_layer; ws holds
   moe_layer_fp8_workspace_bytes(shape) bytes whose header was cleared by
   moe_workspace_init (status word as in include/moe.h). */
size_t moe_layer_fp8_workspace_bytes(const moe_shape* shape);
int moe_layer_fp8(const moe_shape* shape, const uint16_t* x, const uint8_t* xq, const float* xq_scales,
                  const float* w_router, const float* bias, float* logits, const moe_fp8_experts* experts,
                  int32_t* topk_ids, float* topk_w, float* out, void* ws, size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QUANTIZED_ROUTED_MOE_AMD_MOE_FP8_H */
