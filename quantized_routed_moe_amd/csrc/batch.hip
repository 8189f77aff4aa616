// Entry points of the operators of a batch of many requests: argument checks
// (all on the host, before any HIP call) and launches.  See
// include/moe_batch.h for the contract.
#include <algorithm>

#include "../../include/moe_batch.h"
#include "batch.hpp"
#include "validate.hpp"

namespace qrmoe {
namespace {

using check::aligned;

int hip_rc(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

bool known_type(int t) { return t == MOE_TYPE_BF16 || t == MOE_TYPE_F32; }

constexpr int kDimLimit = 1 << 30;
constexpr int kTokenLimit = 1 << 26;
constexpr int64_t kStrideLimit = int64_t{1} << 40;
constexpr int kMostTop = 64;
constexpr int kMostGiven = 4096;

bool batch_ok(int T, int L) { return T >= 0 && T < kTokenLimit && L >= 1 && L <= kMostAdapters; }

bool lora_ok(int T, int K, int N, int r, int L) {
    return batch_ok(T, L) && K >= 32 && K % 32 == 0 && K <= (1 << 22) && N >= 1 && N < kDimLimit && r >= 8 && r % 8 == 0 &&
           r <= 256;
}

constexpr long long kMostBlocks = 1ll << 23;   // of 256 threads or 512: a grid holds fewer than 2^32
constexpr int kMostPolls = 1 << 18;

bool scores_ok(int T, int V, int top) {
    return T >= 0 && T < kDimLimit && V >= 1 && V < kDimLimit && top >= 0 && top <= kMostTop && top <= V;
}

// The parts of either type: what a caller allocates serves both.
size_t scores_ws(int T, int V, int top) {
    const int parts = T ? std::max(score_parts(T, V, true), score_parts(T, V, false)) : 1;
    return parts > 1 ? score_stat_bytes(T, parts) + (static_cast<size_t>(T) * parts * (top + 1) * 8 + 255) / 256 * 256 : 0;
}

int check_ws(const void* ws, size_t ws_bytes, size_t need) {
    if (!need) return MOE_OK;
    if (!ws) return MOE_ERR_NULL;
    if (!aligned(ws, 16)) return MOE_ERR_ALIGN;
    return ws_bytes < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

}  // namespace
}  // namespace qrmoe

using namespace qrmoe;

extern "C" {

size_t moe_lora_items(int32_t T, int32_t L) { return batch_ok(T, L) ? plan_items(T, L) : 0; }

size_t moe_lora_plan_workspace_bytes(int32_t T, int32_t L) { return batch_ok(T, L) ? plan_ws_bytes(T, L) : 0; }

int moe_lora_plan(int32_t T, int32_t L, const int32_t* ids, int32_t* offsets, int32_t* perm, int32_t* items, void* ws,
                  size_t ws_bytes, hipStream_t stream) {
    if (!batch_ok(T, L)) return MOE_ERR_SHAPE;
    if (T == 0) return MOE_OK;
    if (!ids || !offsets || !perm || !items) return MOE_ERR_NULL;
    if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(perm, 4) || !aligned(items, 16)) return MOE_ERR_ALIGN;
    const int rc = check_ws(ws, ws_bytes, plan_ws_bytes(T, L));
    if (rc != MOE_OK) return rc;
    PlanArgs a{T, L, plan_items(T, L), ids, offsets, perm, items, nullptr, nullptr};
    if (T > kPlanBlock) {
        a.first_item = static_cast<int32_t*>(ws);
        a.counts = a.first_item + (L + 1);
    }
    return hip_rc(launch_lora_plan(a, stream));
}

size_t moe_lora_add_workspace_bytes(int32_t T, int32_t K, int32_t N, int32_t r, int32_t L) {
    return lora_ok(T, K, N, r, L) && T ? lora_ws_bytes(lora_shape(T, K, N, r, L), T, r) : 0;
}

int moe_lora_add(int32_t T, int32_t K, int32_t N, int32_t r, int32_t L, const uint16_t* x, int64_t x_stride,
                 const uint16_t* a, const uint16_t* b, const float* scales, const int32_t* perm, const int32_t* items,
                 const void* base, int64_t base_stride, void* out, int64_t out_stride, int32_t type, void* ws,
                 size_t ws_bytes, hipStream_t stream) {
    return moe_lora_add_polls(T, K, N, r, L, x, x_stride, a, b, scales, perm, items, base, base_stride, out, out_stride, type,
                              ws, ws_bytes, kLoraPolls, stream);
}

int moe_lora_add_polls(int32_t T, int32_t K, int32_t N, int32_t r, int32_t L, const uint16_t* x, int64_t x_stride,
                       const uint16_t* a, const uint16_t* b, const float* scales, const int32_t* perm, const int32_t* items,
                       const void* base, int64_t base_stride, void* out, int64_t out_stride, int32_t type, void* ws,
                       size_t ws_bytes, int32_t polls, hipStream_t stream) {
    if (!lora_ok(T, K, N, r, L) || polls < 0 || polls > kMostPolls) return MOE_ERR_SHAPE;
    if (T == 0) return MOE_OK;
    if (!x || !a || !b || !perm || !items || !base || !out) return MOE_ERR_NULL;
    if (!known_type(type)) return MOE_ERR_FORMAT;
    if (x_stride % 8 || x_stride < 0 || (x_stride && x_stride < K) || x_stride > kStrideLimit) return MOE_ERR_SHAPE;
    if (base_stride < 0 || (base_stride && base_stride < N) || base_stride > kStrideLimit) return MOE_ERR_SHAPE;
    if (out_stride < N || out_stride > kStrideLimit) return MOE_ERR_SHAPE;
    if (base == out && base_stride != out_stride) return MOE_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(base, 16) || !aligned(out, 16) ||
        !aligned(items, 16) || !aligned(perm, 4) || !aligned(scales, 4))
        return MOE_ERR_ALIGN;
    const LoraShape shape = lora_shape(T, K, N, r, L);
    if (shape.blocks >= kMostBlocks) return MOE_ERR_SHAPE;
    const int rc = check_ws(ws, ws_bytes, lora_ws_bytes(shape, T, r));
    if (rc != MOE_OK) return rc;
    LoraArgs p{};
    p.T = T;
    p.K = K;
    p.N = N;
    p.r = r;
    p.L = L;
    p.n_items = plan_items(T, L);
    p.x = x;
    p.x_stride = x_stride;
    p.a = a;
    p.b = b;
    p.scales = scales;
    p.perm = perm;
    p.items = items;
    p.base = base;
    p.out = out;
    p.base_stride = base_stride;
    p.out_stride = out_stride;
    p.f32 = type == MOE_TYPE_F32;
    const int per = p.f32 ? 4 : 8;
    p.vec = N % 8 == 0 && base_stride % per == 0 && out_stride % per == 0;
    p.in_place = base == out;
    p.splits = shape.splits;
    p.v = static_cast<float*>(ws);
    p.flags = reinterpret_cast<unsigned long long*>(static_cast<char*>(ws) + lora_v_bytes(shape, T, r));
    p.polls = polls;
    return hip_rc(launch_lora_add(p, stream));
}

size_t moe_token_logprobs_workspace_bytes(int32_t T, int32_t V, int32_t top) {
    return scores_ok(T, V, top) ? scores_ws(T, V, top) : 0;
}

int moe_token_logprobs(int32_t T, int32_t V, const void* logits, int32_t type, int64_t stride, const int32_t* tokens,
                       int32_t given, float* logprobs, float* entropy, int32_t top, int32_t* top_ids,
                       float* top_logprobs, void* ws, size_t ws_bytes, hipStream_t stream) {
    if (!scores_ok(T, V, top) || given < 0 || given > kMostGiven) return MOE_ERR_SHAPE;
    if (T == 0) return MOE_OK;
    if (!logits || (given && (!tokens || !logprobs)) || (top && (!top_ids || !top_logprobs))) return MOE_ERR_NULL;
    if (!given && !top && !entropy) return MOE_ERR_NULL;
    if (!known_type(type)) return MOE_ERR_FORMAT;
    if (stride < V || stride > kStrideLimit) return MOE_ERR_SHAPE;
    if (!aligned(logits, 16) || !aligned(tokens, 4) || !aligned(logprobs, 4) || !aligned(entropy, 4) || !aligned(top_ids, 4) ||
        !aligned(top_logprobs, 4))
        return MOE_ERR_ALIGN;
    const int rc = check_ws(ws, ws_bytes, scores_ws(T, V, top));
    if (rc != MOE_OK) return rc;
    const bool f32 = type == MOE_TYPE_F32;
    const int parts = score_parts(T, V, f32);
    ScoreArgs p{T, V, given, top, parts, score_take(T, V, top, f32, parts), logits, stride, tokens, logprobs, entropy, top_logprobs, top_ids,
                nullptr, nullptr, nullptr};
    if (p.parts > 1) {
        p.stats = static_cast<float*>(ws);
        p.flags = reinterpret_cast<unsigned long long*>(static_cast<char*>(ws) + score_stat_bytes(T, p.parts));
        p.keys = p.flags + static_cast<size_t>(T) * p.parts;
    }
    return hip_rc(launch_scores(p, f32, stream));
}

}  // extern "C"
