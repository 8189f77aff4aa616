// Shared parts of the operators of a batch of many requests
// (include/moe_batch.h): kernel arguments, sizes and the launch interface
// between the entry points (batch.hip) and the kernels.
#pragma once

#include "common.hpp"

namespace qrmoe {

constexpr int kMostAdapters = 1024;
constexpr int kItemRows = 64;                  // tokens of one run of the schedule

// ---- plan

constexpr int kPlanBlock = 8192;               // tokens that one workgroup sorts

struct PlanArgs {
    int T, L, n_items;
    const int32_t* ids;
    int32_t *offsets, *perm, *items;
    int32_t* counts;                           // T > kPlanBlock: [blocks][L+1] tokens of a block and group, then
                                               // their place among the group's tokens
    int32_t* first_item;                       // [L+1]
};

inline int plan_items(int T, int L) {
    const long long groups = L + 1 < T ? L + 1 : T;
    return static_cast<int>((T + groups * (kItemRows - 1)) / kItemRows);       // each group's last run as short as can be
}
inline size_t plan_blocks(int T) { return (static_cast<size_t>(T) + kPlanBlock - 1) / kPlanBlock; }
inline size_t plan_ws_bytes(int T, int L) {
    return T <= kPlanBlock ? 0 : ((plan_blocks(T) + 1) * (L + 1) * 4 + 255) / 256 * 256;
}

hipError_t launch_lora_plan(const PlanArgs& a, hipStream_t st);

// ---- adapters

// How a call is cut into workgroups (lora.hip).
struct LoraShape {
    int splits;                                // parts of K; 0: few tokens, no workspace
    long long flags;                           // workgroups that make v, one flag each
    long long blocks;                          // all
};
LoraShape lora_shape(int T, int K, int N, int r, int L);
inline size_t lora_v_bytes(const LoraShape& p, int T, int r) { return (static_cast<size_t>(p.splits) * T * r * 4 + 255) / 256 * 256; }
inline size_t lora_ws_bytes(const LoraShape& p, int T, int r) { return lora_v_bytes(p, T, r) + (p.flags * 8 + 255) / 256 * 256; }

struct LoraArgs {
    int T, K, N, r, L, n_items;
    const uint16_t* x;
    long long x_stride;
    const uint16_t *a, *b;
    const float* scales;
    const int32_t *perm, *items;
    const void* base;
    void* out;
    long long base_stride, out_stride;
    int f32;                                   // 1: base and out are fp32, 0: bf16
    int vec;                                   // 1: eight columns of base and out lie in whole 16 bytes, N is a multiple of 8
    int in_place;
    int splits;
    float* v;                                  // [splits][T][r], by entry of perm
    unsigned long long* flags;
    int polls;                                 // of a wait for v, 0: none
    int tid;                                   // of the kernel: threadIdx.x
};

// About 20 ms, far beyond what v of one run takes (K of 2^22: 1 ms), and a sixteenth of
// the layer's bound: what waits here makes room before a layer beside it gives up.
constexpr int kLoraPolls = 1 << 14;

hipError_t launch_lora_add(const LoraArgs& a, hipStream_t st);

// ---- scores

// What a workgroup takes (scores.hip).
enum class ScoreTake {
    kRows,   // a row a wave
    kRow,    // a row
    kPart    // a part of a row, or a short one, seen twice
};

struct ScoreArgs {
    int T, V, given, top, parts;
    ScoreTake take;
    const void* logits;
    long long stride;
    const int32_t* tokens;
    float *logprobs, *entropy, *top_logprobs;
    int32_t* top_ids;
    float* stats;                              // parts > 1: [T][parts][4] maximum, sum, weighted sum
    unsigned long long* keys;                  // [T][parts][top]
    unsigned long long* flags;                 // [T][parts]
};

int score_parts(int T, int V, bool f32);       // at most 32
ScoreTake score_take(int T, int V, int top, bool f32, int parts);
inline size_t score_stat_bytes(int T, int parts) { return (static_cast<size_t>(T) * parts * 16 + 255) / 256 * 256; }

hipError_t launch_scores(const ScoreArgs& a, bool f32, hipStream_t st);

}  // namespace qrmoe
