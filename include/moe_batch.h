/*
 * moe_batch.h -- C ABI of the operators of a batch of many requests, beside
 * the FP8 operators of include/moe_fp8.h, for AMD Instinct MI355X (gfx950).
 *
 * A serving step runs the tokens of many requests through one set of
 * weights.  What differs from request to request is here: the low-rank
 * adapter that a request adds to a shared projection, and what a request
 * wants to know of its row of logits.  The chain: moe_add_rmsnorm makes bf16
 * rows and E4M3 rows; moe_gemm_fp8 is the shared projection of the E4M3 rows;
 * moe_lora_add adds to its result the adapters' part of the bf16 rows; after
 * the product with the vocabulary, moe_token_logprobs reads the logits (of
 * the drafted tokens of a verify step, of a prompt, of the sampled tokens).
 *
 * Conventions as in include/moe.h: device pointers, caller-owned buffers, no
 * allocation, every call only enqueues on `stream` (a stream of the current
 * device), host-side validation before any HIP call, negative status codes
 * (enum moe_status).  Calls are independent: nothing is kept between them.
 * Every call may be captured into a HIP graph.  Results do not depend on
 * timing: no floating-point atomics, sums in a fixed order.
 *
 * Alignment: x, a, b, base, out, logits, items and ws 16 bytes; other arrays
 * 4 bytes.  Inputs and outputs must not overlap except where stated.
 */
#ifndef QUANTIZED_ROUTED_MOE_AMD_MOE_BATCH_H
#define QUANTIZED_ROUTED_MOE_AMD_MOE_BATCH_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#include "moe.h"
#include "moe_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Groups a batch's tokens by adapter, once for all projections of a step.
   ids int32 [T]: the adapter of each token, in [0, L); a token with any
   other id has none and belongs to group L.

     perm int32 [T]       the tokens by group, those of a group in order
     offsets int32 [L+2]  group g's tokens are perm[offsets[g] .. offsets[g+1])
     items int32 [moe_lora_items(T, L)][4]
                          the schedule of moe_lora_add: (group, first, end, 0)
                          of runs of at most 64 entries of perm, by group;
                          past the last run (-1, 0, 0, 0)

   ws: moe_lora_plan_workspace_bytes(T, L) bytes (0: ws may be NULL),
   uninitialised; one call at a time.  T == 0 enqueues nothing.
   Limits: 0 <= T < 2^26, 1 <= L <= 1024 (moe_lora_items and
   moe_lora_plan_workspace_bytes return 0 outside them).  Errors:
   MOE_ERR_SHAPE, MOE_ERR_NULL, MOE_ERR_ALIGN, MOE_ERR_WORKSPACE, MOE_ERR_HIP. */
size_t moe_lora_items(int32_t T, int32_t L);
size_t moe_lora_plan_workspace_bytes(int32_t T, int32_t L);
int moe_lora_plan(int32_t T, int32_t L, const int32_t* ids, int32_t* offsets, int32_t* perm, int32_t* items, void* ws,
                  size_t ws_bytes, hipStream_t stream);

/* Low-rank adapters of many requests beside a shared projection of T rows of
   K values to N columns: for token t of adapter g

     v[j]      = sum_k x[t][k] * a[g][j][k]                             (fp32)
     out[t][n] = base[t][n] + scales[g] * sum_j v[j] * b[g][n][j]       (fp32, rounded once to `type`)

   and out[t] = base[t] for a token of no adapter.
   x bf16 [T][K], rows x_stride values apart (a multiple of 8, >= K; or 0,
   one row for all); a bf16 [L][r][K]; b bf16 [L][N][r]; scales fp32 [L] or
   NULL (1); perm, items: of moe_lora_plan for T and L.  base, out: `type`
   (MOE_TYPE_BF16 or MOE_TYPE_F32) [T][N], rows base_stride (0, one row for
   all, or >= N) and out_stride (>= N) values apart; out may be base itself (in
   place, same stride), whose rows of no adapter are then not touched.
   Both sums have the accuracy of fp32 sums of exact products whatever
   `type`, but for what lies below 2^-126: a product that small, and in a v
   below 2^-102 the bits that are, may count as 0.  A value of v that is not finite (or not below 2^128 - 2^119) makes
   its token's row non-finite, one of b its column of its adapter's tokens.
   A rank that is no multiple of 8 is padded with zero rows of a and columns
   of b.  Adapters without tokens are not read.  Entries of perm and items
   outside their ranges are skipped, never followed.
   ws: moe_lora_add_workspace_bytes(T, K, N, r, L) bytes (0, with few tokens:
   ws may be NULL), uninitialised; one call at a time.  It holds v, which
   workgroups hand to others of the same launch by flags; one that waits for a
   flag longer than about 20 ms (launches on several streams can keep each
   other's workgroups from their places) makes the v it needs itself, so the
   result does not depend on it.  T == 0 enqueues nothing.
   moe_lora_add_polls: the same, with the number of times a workgroup asks for
   a flag, from 0 (it makes v itself at once) to 2^18, else MOE_ERR_SHAPE.  The
   result has the same bits; moe_lora_add takes 2^14.
   Limits: T and L as moe_lora_plan; K a positive multiple of 32 up to 2^22;
   1 <= N < 2^30; r a multiple of 8 from 8 to 256; fewer than 2^23 workgroups:
   two per item for each 512 columns, and two per item, 32 ranks and part of K
   (1, 2, 4 or 8 of them, one with many tokens), items * 2 rounded up to 16.
   Errors: MOE_ERR_SHAPE, MOE_ERR_NULL,
   MOE_ERR_FORMAT (type), MOE_ERR_ALIGN, MOE_ERR_WORKSPACE,
   MOE_ERR_UNSUPPORTED (out is base with another stride), MOE_ERR_HIP. */
size_t moe_lora_add_workspace_bytes(int32_t T, int32_t K, int32_t N, int32_t r, int32_t L);
int moe_lora_add(int32_t T, int32_t K, int32_t N, int32_t r, int32_t L, const uint16_t* x, int64_t x_stride,
                 const uint16_t* a, const uint16_t* b, const float* scales, const int32_t* perm, const int32_t* items,
                 const void* base, int64_t base_stride, void* out, int64_t out_stride, int32_t type, void* ws,
                 size_t ws_bytes, hipStream_t stream);
int moe_lora_add_polls(int32_t T, int32_t K, int32_t N, int32_t r, int32_t L, const uint16_t* x, int64_t x_stride,
                       const uint16_t* a, const uint16_t* b, const float* scales, const int32_t* perm, const int32_t* items,
                       const void* base, int64_t base_stride, void* out, int64_t out_stride, int32_t type, void* ws,
                       size_t ws_bytes, int32_t polls, hipStream_t stream);

/* Log probabilities of rows of logits l [V] (log p_v = l_v - log sum e^l):

     logprobs[t][i]     = log p of tokens[t][i]
     entropy[t]         = - sum_v p_v log p_v
     top_ids[t][j]      the `top` likeliest tokens in order, ties to the lower id
     top_logprobs[t][j] = log p of them

   logits: `type` (MOE_TYPE_BF16 or MOE_TYPE_F32) [T][V], rows stride values
   apart (>= V); any row may start at a multiple of its value's size.
   tokens int32 [T][given] with logprobs fp32 [T][given] (given = 0: both
   may be NULL); entropy fp32 [T] or NULL; top_ids int32 and top_logprobs
   fp32 [T][top] (top = 0: both may be NULL); at least one output.  Sums are
   fp32.
   A logit of -inf has probability 0 and log probability -inf, and stands
   behind all others in the order.  A row with nothing but -inf: every log
   probability is -inf, the entropy 0.  A row holding a NaN or +inf: its
   floats are NaN, its top_ids -1.  A token outside [0, V) is not followed:
   its log probability is NaN.
   ws: moe_token_logprobs_workspace_bytes(T, V, top) bytes (0, with many rows or
   short ones: ws may be NULL), uninitialised; one call at a time.  It holds the
   results of parts of a row, which the workgroup that finds them all there
   joins; none waits for another.  T == 0 enqueues nothing.
   Limits: 0 <= T < 2^30, 1 <= V < 2^30, 0 <= given <= 4096, 0 <= top <=
   min(V, 64).  Errors: MOE_ERR_SHAPE, MOE_ERR_NULL, MOE_ERR_FORMAT (type),
   MOE_ERR_ALIGN, MOE_ERR_WORKSPACE, MOE_ERR_HIP. */
size_t moe_token_logprobs_workspace_bytes(int32_t T, int32_t V, int32_t top);
int moe_token_logprobs(int32_t T, int32_t V, const void* logits, int32_t type, int64_t stride, const int32_t* tokens,
                       int32_t given, float* logprobs, float* entropy, int32_t top, int32_t* top_ids,
                       float* top_logprobs, void* ws, size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QUANTIZED_ROUTED_MOE_AMD_MOE_BATCH_H */
