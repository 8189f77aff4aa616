// Groups a batch's tokens by adapter (moe_lora_plan): a stable counting sort
// by group (group L: no adapter), and the schedule of the adapter kernels, runs
// of at most 64 tokens of one group.
//
// Reads 4 T bytes and writes 4 T and the schedule: bound by the launch and a
// chain of LDS round trips (64 tokens 3.0 us, of which a launch that does nothing is
// 2.2; 8192 of 256 adapters 9.7; 65536 20), and done once a batch for all its projections.
// Up to kPlanBlock tokens in one workgroup; beyond, three launches: counts of
// every block of tokens, their places by a scan over the blocks, and the sort
// of each block into its places.
//
// Tokens of one group within a wave's 64: the AND of the group's bits' ballots;
// a token's place is the count of lower lanes among them.  Waves take consecutive
// tokens and count into rows of their own, so nothing depends on the order of
// atomics.
#include "batch.hpp"

namespace qrmoe {

namespace {

constexpr int kMostGroups = kMostAdapters + 1;

__device__ __forceinline__ int group_of(const PlanArgs& a, int t) {
    const int id = a.ids[t];
    return id >= 0 && id < a.L ? id : a.L;
}

// Groups of a wave's 64 * ROUNDS consecutive tokens from t0 on; -1 past the last.
template <int ROUNDS>
__device__ __forceinline__ void load_groups(const PlanArgs& a, int t0, int (&group)[ROUNDS]) {
#pragma unroll
    for (int j = 0; j < ROUNDS; ++j) {
        const int t = t0 + 64 * j + static_cast<int>(threadIdx.x & 63);
        const int g = group_of(a, min(t, a.T - 1));
        group[j] = t < a.T ? g : -1;
    }
}

// Their ranks among the wave's tokens of their group, and the wave's counts in
// cnt[group].
template <int ROUNDS>
__device__ __forceinline__ void rank_wave(const int (&group)[ROUNDS], volatile int* cnt, int bits, int (&rank)[ROUNDS]) {
    const int lane = threadIdx.x & 63;
    const uint64_t below = lane ? ~0ull >> (64 - lane) : 0ull;
    // lanes that differ, in halves: a bit's ballot, turned round where the lane's is set
    uint32_t lo[ROUNDS], hi[ROUNDS];
#pragma unroll
    for (int j = 0; j < ROUNDS; ++j) lo[j] = hi[j] = 0u;
    for (int b = 0; b < bits; ++b)
#pragma unroll
        for (int j = 0; j < ROUNDS; ++j) {
            const uint32_t mine = static_cast<uint32_t>(static_cast<int>(static_cast<uint32_t>(group[j]) << (31 - b)) >> 31);
            const uint64_t ones = __ballot(mine != 0u);
            lo[j] |= static_cast<uint32_t>(ones) ^ mine;
            hi[j] |= static_cast<uint32_t>(ones >> 32) ^ mine;
        }
#pragma unroll
    for (int j = 0; j < ROUNDS; ++j) {
        const int g = group[j];
        const uint64_t there = __ballot(g >= 0);
        const uint64_t same = ~(static_cast<uint64_t>(hi[j]) << 32 | lo[j]) & (g >= 0 ? there : ~there);
        // every lane reads before the group's highest lane writes: one wave,
        // whose LDS accesses are in order
        const int before = g >= 0 ? cnt[g] : 0;
        rank[j] = before + __popcll(same & below);
        if (g >= 0 && same >> lane == 1ull) cnt[g] = before + __popcll(same);
    }
}

// Exclusive scans of v over the workgroup's threads; total: in every thread.
template <int WAVES>
__device__ __forceinline__ int2 block_scan(int2 v, int2* part, int2& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int2 incl = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int x = __shfl_up(incl.x, o), y = __shfl_up(incl.y, o);
        if (lane >= o) {
            incl.x += x;
            incl.y += y;
        }
    }
    if (lane == 63) part[wave] = incl;
    __syncthreads();
    int2 base = make_int2(0, 0), sum = make_int2(0, 0);
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        const int2 p = part[w];
        if (w < wave) {
            base.x += p.x;
            base.y += p.y;
        }
        sum.x += p.x;
        sum.y += p.y;
    }
    total = sum;
    return make_int2(base.x + incl.x - v.x, base.y + incl.y - v.y);
}

__device__ __forceinline__ void store_item(const PlanArgs& a, int at, int g, int first, int end) {
    reinterpret_cast<int4*>(a.items)[at] = make_int4(g, first, end, 0);
}

__device__ __forceinline__ int item_count(int tokens) { return (tokens + kItemRows - 1) / kItemRows; }

// Offsets and first items of the groups from their totals in LDS, which they
// replace; unused items.  All threads; PER consecutive groups a thread.
template <int WAVES>
__device__ __forceinline__ void scan_groups(const PlanArgs& a, int* tokens, int* first_item, int2* part) {
    const int G = a.L + 1, per = (G + WAVES * 64 - 1) / (WAVES * 64);
    const int g0 = min(static_cast<int>(threadIdx.x) * per, G), g1 = min(g0 + per, G);
    int2 n = make_int2(0, 0), all;             // tokens and items
    for (int g = g0; g < g1; ++g) {
        n.x += tokens[g];
        n.y += item_count(tokens[g]);
    }
    const int2 before = block_scan<WAVES>(n, part, all);
    int at = before.x, item = before.y;
    for (int g = g0; g < g1; ++g) {
        const int c = tokens[g];
        tokens[g] = at;
        a.offsets[g] = at;
        first_item[g] = item;
        at += c;
        item += item_count(c);
    }
    if (threadIdx.x == 0) {
        tokens[G] = all.x;
        a.offsets[G] = all.x;
    }
    for (int i = all.y + threadIdx.x; i < a.n_items; i += WAVES * 64) store_item(a, i, -1, 0, 0);
}

// Up to WAVES * ROUNDS * 64 tokens.
template <int WAVES, int ROUNDS>
__global__ __launch_bounds__(WAVES* kWave) void plan_kernel(PlanArgs a, int bits) {
    __shared__ int cnt[WAVES * kMostGroups];   // [WAVES][G], then each wave's first place in the group
    __shared__ int start[kMostGroups + 1], first_item[kMostGroups];
    __shared__ int2 part[WAVES];
    __shared__ int sorted[WAVES * ROUNDS * kWave];             // perm, from where it is written in order
    const int G = a.L + 1, wave = threadIdx.x >> 6;
    int group[ROUNDS], rank[ROUNDS];
    const int t0 = wave * ROUNDS * kWave;
    load_groups(a, t0, group);
    for (int i = threadIdx.x; i < WAVES * G; i += WAVES * kWave) cnt[i] = 0;
    __syncthreads();
    rank_wave(group, cnt + wave * G, bits, rank);
    __syncthreads();
    for (int g = threadIdx.x; g < G; g += WAVES * kWave) {
        int sum = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const int c = cnt[w * G + g];
            cnt[w * G + g] = sum;
            sum += c;
        }
        start[g] = sum;
    }
    __syncthreads();
    scan_groups<WAVES>(a, start, first_item, part);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < ROUNDS; ++j) {
        const int g = group[j];
        if (g < 0) continue;
        const int in_group = cnt[wave * G + g] + rank[j], at = start[g] + in_group;
        sorted[at] = t0 + 64 * j + (threadIdx.x & 63);
        if (in_group % kItemRows == 0)
            store_item(a, first_item[g] + in_group / kItemRows, g, at, min(at + kItemRows, start[g + 1]));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.T; i += WAVES * kWave) a.perm[i] = sorted[i];
}

constexpr int kBlockWaves = 16, kBlockRounds = kPlanBlock / (kBlockWaves * kWave);

// Tokens of each group in a block of kPlanBlock.
__global__ __launch_bounds__(kBlockWaves* kWave) void plan_count_kernel(PlanArgs a) {
    __shared__ int lds[kMostGroups];
    const int G = a.L + 1;
    for (int i = threadIdx.x; i < G; i += blockDim.x) lds[i] = 0;
    __syncthreads();
    const long long t0 = static_cast<long long>(blockIdx.x) * kPlanBlock;
    for (int i = threadIdx.x; i < kPlanBlock && t0 + i < a.T; i += blockDim.x) atomicAdd(lds + group_of(a, static_cast<int>(t0 + i)), 1);
    __syncthreads();
    for (int g = threadIdx.x; g < G; g += blockDim.x) a.counts[static_cast<size_t>(blockIdx.x) * G + g] = lds[g];
}

// One workgroup: a block's counts become its first places in the groups.
__global__ __launch_bounds__(kBlockWaves* kWave) void plan_scan_kernel(PlanArgs a, int blocks) {
    __shared__ int start[kMostGroups + 1], first_item[kMostGroups];
    __shared__ int2 part[kBlockWaves];
    constexpr int kAhead = 16;                 // counts on their way at a time
    const int G = a.L + 1;
    for (int g = threadIdx.x; g < G; g += blockDim.x) {
        int sum = 0;
        for (int b = 0; b < blocks; b += kAhead) {
            int* p = a.counts + static_cast<size_t>(b) * G + g;
            int c[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) c[i] = b + i < blocks ? p[static_cast<size_t>(i) * G] : 0;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (b + i < blocks) p[static_cast<size_t>(i) * G] = sum;
                sum += c[i];
            }
        }
        start[g] = sum;
    }
    __syncthreads();
    scan_groups<kBlockWaves>(a, start, first_item, part);
    __syncthreads();
    for (int g = threadIdx.x; g < G; g += blockDim.x) a.first_item[g] = first_item[g];
}

__global__ __launch_bounds__(kBlockWaves* kWave) void plan_place_kernel(PlanArgs a, int bits) {
    __shared__ int lds[kBlockWaves * kMostGroups];     // as plan_kernel's cnt
    const int G = a.L + 1, wave = threadIdx.x >> 6;
    int group[kBlockRounds], rank[kBlockRounds];
    const int t0 = blockIdx.x * kPlanBlock + wave * kBlockRounds * kWave;
    load_groups(a, t0, group);
    for (int i = threadIdx.x; i < kBlockWaves * G; i += blockDim.x) lds[i] = 0;
    __syncthreads();
    rank_wave(group, lds + wave * G, bits, rank);
    __syncthreads();
    for (int g = threadIdx.x; g < G; g += blockDim.x) {
        int sum = a.counts[static_cast<size_t>(blockIdx.x) * G + g];
#pragma unroll
        for (int w = 0; w < kBlockWaves; ++w) {
            const int c = lds[w * G + g];
            lds[w * G + g] = sum;
            sum += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kBlockRounds; ++j) {
        const int g = group[j];
        if (g < 0) continue;
        const int in_group = lds[wave * G + g] + rank[j], at = a.offsets[g] + in_group;
        a.perm[at] = t0 + 64 * j + (threadIdx.x & 63);
        if (in_group % kItemRows == 0)
            store_item(a, a.first_item[g] + in_group / kItemRows, g, at, min(at + kItemRows, a.offsets[g + 1]));
    }
}

}  // namespace

hipError_t launch_lora_plan(const PlanArgs& a, hipStream_t st) {
    int bits = 1;
    while (a.L >> bits) ++bits;
    if (a.T <= kPlanBlock) {
        // us: 64 tokens 3.0 (300 in sixteen waves 4.3); 300 in two rounds 4.3, in eight 6.7; 2048 4.6, 7.2
        if (a.T <= 256) plan_kernel<4, 1><<<1, 4 * kWave, 0, st>>>(a, bits);
        else if (a.T <= 2048) plan_kernel<kBlockWaves, 2><<<1, kBlockWaves * kWave, 0, st>>>(a, bits);
        else plan_kernel<kBlockWaves, kBlockRounds><<<1, kBlockWaves * kWave, 0, st>>>(a, bits);
        return hipGetLastError();
    }
    const int blocks = static_cast<int>(plan_blocks(a.T));
    plan_count_kernel<<<blocks, kBlockWaves * kWave, 0, st>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    plan_scan_kernel<<<1, kBlockWaves * kWave, 0, st>>>(a, blocks);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    plan_place_kernel<<<blocks, kBlockWaves * kWave, 0, st>>>(a, bits);
    return hipGetLastError();
}

}  // namespace qrmoe
