// Log probabilities of rows of logits (moe_token_logprobs): for every row the
// maximum m, S = sum e^(l - m), U = sum e^(l - m) (l - m) and the largest `top`
// logits in one pass; then log p = l - m - ln S, the entropy ln S - U / S.
//
// Bound by HBM with many rows (each logit is read once), by latency with few:
// a row is then cut into parts, whose results a second launch joins.
//
// A wave takes 16 bytes a lane and chunk, four chunks ahead of their use, and
// holds m, S and U for each lane apart, corrected once per round of chunks if the
// lane's maximum rose; the lanes meet at the end.  The wave's largest logits are a
// list sorted over its lanes (key: value, then lowest place).  A chunk whose
// largest value is not above the list's last takes one comparison; the others'
// values enter one by one.  The first round's list would take a value at a
// time, so it begins at a bound: the top-th largest of the lanes' maxima, below which
// none of the row's top can be.
//
// Logits of -inf are kept out of the lists (a masked vocabulary would fill them
// again and again): a row with fewer than `top` others takes the lowest places of
// -inf at the end.
#include "batch.hpp"
#include "topk_dev.hpp"

namespace qrmoe {

namespace {

constexpr int kScoreWaves = 4;
constexpr int kScoreThreads = kScoreWaves * kWave;
constexpr float kLowest = -3.402823466e38f;    // the lowest finite float
constexpr float kFar = -1e30f;                 // e^kFar is 0, and kFar times a sum is finite
constexpr float kLog2e = 1.44269504088896341f;

typedef unsigned long long Key;                // float_key(value) << 32 | ~place; 0: none

__device__ __forceinline__ Key make_key(float v, uint32_t place) {
    return static_cast<Key>(float_key(v)) << 32 | (0xffffffffu - place);
}
__device__ __forceinline__ uint32_t key_place(Key k) { return 0xffffffffu - static_cast<uint32_t>(k); }
__device__ __forceinline__ float key_value(Key k) {
    const uint32_t u = static_cast<uint32_t>(k >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ Key key_of_lane(Key k, int lane) {
    const int lo = lane_value(static_cast<int>(static_cast<uint32_t>(k)), lane);
    const int hi = lane_value(static_cast<int>(static_cast<uint32_t>(k >> 32)), lane);
    return static_cast<Key>(static_cast<uint32_t>(hi)) << 32 | static_cast<uint32_t>(lo);
}

// The list of a wave: lane i holds the i-th largest key of those seen.
struct TopList {
    Key mine = 0;
    Key last = 0;                              // lane top - 1's
    float bound = kLowest;                     // values below it need no look

    __device__ __forceinline__ void refresh(int top) {
        last = key_of_lane(mine, top - 1);
        if (last) bound = fmaxf(bound, key_value(last));
    }
    // k > last, uniform
    __device__ __forceinline__ void insert(Key k, int top) {
        const int lane = threadIdx.x & 63;
        const int at = __popcll(__ballot(mine > k));
        const Key up = __shfl_up(mine, 1);
        mine = lane < at ? mine : lane == at ? k : up;
        refresh(top);
    }
    // Values v of the lanes (place: each lane's) that are not below the bound.
    __device__ __forceinline__ void offer(float v, uint32_t place, int top) {
        const Key k = make_key(v, place);
        bool in = v >= bound && k > last;
        for (uint64_t mask = __ballot(in); mask; mask = __ballot(in)) {
            const int from = __ffsll(static_cast<unsigned long long>(mask)) - 1;
            insert(key_of_lane(k, from), top);
            in = in && k > last && static_cast<int>(threadIdx.x & 63) != from;
        }
    }
    // With another sorted list: the larger of one list's i-th and the other's
    // i-th from the end are the 64 largest, rising and falling once, which six
    // exchanges sort.
    __device__ __forceinline__ void merge(Key other) {
        const int lane = threadIdx.x & 63;
        const Key turned = __shfl(other, 63 - lane);
        mine = mine > turned ? mine : turned;
#pragma unroll
        for (int o = 32; o; o >>= 1) {
            const Key there = __shfl_xor(mine, o);
            const bool take = lane & o ? there < mine : there > mine;
            mine = take ? there : mine;
        }
    }
};

struct Stats {
    float m = -INFINITY, s = 0.f, u = 0.f;

    static __device__ __forceinline__ Stats of(const float* p) {
        Stats r;
        r.m = p[0];
        r.s = p[1];
        r.u = p[2];
        return r;
    }
    __device__ __forceinline__ void store(float* p) const {
        p[0] = m;
        p[1] = s;
        p[2] = u;
    }
    // Sums relative to a maximum `to` >= m.
    __device__ __forceinline__ void raise(float to) {
        const float d = to > m ? fmaxf(m - to, kFar) : 0.f;
        const float c = __builtin_amdgcn_exp2f(d * kLog2e);
        u = c * fmaf(s, d, u);
        s *= c;
        m = to;
    }
    template <bool ENT>
    __device__ __forceinline__ void add(float l, float at) {
        const float d = l - at;
        const float e = __builtin_amdgcn_exp2f(d * kLog2e);
        s += e;
        if constexpr (ENT) u = fmaf(e, fmaxf(d, kFar), u);        // 0 times a finite value where l is -inf
    }
    __device__ __forceinline__ void join(const Stats& o) {
        const float to = fmaxf(m, o.m);
        Stats b = o;
        raise(to);
        b.raise(to);
        s += b.s;
        u += b.u;
    }
};

__device__ __forceinline__ float finite_or_zero(float m) { return m == -INFINITY ? 0.f : m; }

template <bool F32>
__device__ __forceinline__ float logit_at(const void* row, long long i) {
    if constexpr (F32) return static_cast<const float*>(row)[i];
    else return bf16_to_f32(static_cast<const uint16_t*>(row)[i]);
}

// The top-th largest of the lanes' values, by counting for each those before it.
__device__ __forceinline__ float nth_of_lanes(float v, int top) {
    const int lane = threadIdx.x & 63;
    int before = 0;
#pragma unroll
    for (int j = 0; j < 64; ++j) {
        const float o = lane_value(v, j);
        before += o > v || (o == v && j < lane);
    }
    const uint64_t hit = __ballot(before == top - 1);
    return lane_value(v, __ffsll(static_cast<unsigned long long>(hit)) - 1);
}

// Outputs of row t from its statistics and list, by one wave.
template <bool F32>
__device__ __forceinline__ void finish_row(const ScoreArgs& a, int t, const void* row, Stats st, TopList list) {
    const int lane = threadIdx.x & 63;
    const float m = finite_or_zero(st.m), ln_s = logf(st.s);      // all -inf: m 0, ln 0 = -inf; NaN if a logit was NaN or +inf
    const bool empty = st.s == 0.f;
    auto logprob = [&](float l) { return empty ? -INFINITY : (l - m) - ln_s; };
    if (a.entropy && lane == 0) a.entropy[t] = empty ? 0.f : ln_s - st.u / st.s;
    for (int i = lane; i < a.given; i += 64) {
        const size_t at = static_cast<size_t>(t) * a.given + i;
        const int tok = a.tokens[at];
        float lp = NAN;
        if (tok >= 0 && tok < a.V && st.s == st.s) lp = logprob(logit_at<F32>(row, tok));
        a.logprobs[at] = lp;
    }
    if (!a.top) return;
    // places of -inf in order, if the others do not fill the list: they are
    // fewer than top, so the first 128 places hold enough
    int found = __popcll(__ballot(list.mine != 0));
    for (int i0 = 0; st.s == st.s && found < a.top && i0 < a.V; i0 += 64) {
        const int i = i0 + lane;
        const uint64_t hidden = __ballot(i < a.V && logit_at<F32>(row, min(i, a.V - 1)) == -INFINITY);
        for (uint64_t left = hidden; left && found < a.top; left &= left - 1) {
            const int from = __ffsll(static_cast<unsigned long long>(left)) - 1;
            if (lane == found) list.mine = make_key(-INFINITY, i0 + from);
            ++found;
        }
    }
    if (lane < a.top) {
        const size_t at = static_cast<size_t>(t) * a.top + lane;
        const bool bad = st.s != st.s || !list.mine;
        a.top_ids[at] = bad ? -1 : static_cast<int>(key_place(list.mine));
        a.top_logprobs[at] = bad ? NAN : logprob(key_value(list.mine));
    }
}

template <bool F32, bool ENT, bool TOP>
__global__ __launch_bounds__(kScoreThreads) void scores_kernel(ScoreArgs a, int t0) {
    constexpr int kPer = F32 ? 4 : 8, kAhead = 4;              // values of a chunk, chunks of a round
    __shared__ float stats[kScoreWaves][3];
    __shared__ Key keys[kScoreWaves][kWave];
    const int part = blockIdx.x % a.parts, t = t0 + blockIdx.x / a.parts;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const char* row = static_cast<const char*>(a.logits) + t * a.stride * (F32 ? 4 : 2);
    // values before the first whole 16 bytes, whole chunks, values after
    const int head = min(static_cast<int>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (F32 ? 4 : 2), a.V);
    const int chunks = (a.V - head) / kPer, body = head + chunks * kPer;
    const u32x4* data = reinterpret_cast<const u32x4*>(row + head * (F32 ? 4 : 2));
    const int c_beg = static_cast<int>(static_cast<long long>(chunks) * part / a.parts);
    const int c_end = static_cast<int>(static_cast<long long>(chunks) * (part + 1) / a.parts);

    Stats st;
    TopList list;
    bool first = true;
    auto values = [&](u32x4 w, float (&v)[kPer]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (F32) {
                v[i] = __uint_as_float(w[i]);
            } else {
                v[2 * i] = bf16lo(w[i]);
                v[2 * i + 1] = bf16hi(w[i]);
            }
        }
    };
    constexpr int kRound = kAhead * kWave;
    for (int c0 = c_beg + wave * kRound; c0 < c_end; c0 += kScoreWaves * kRound) {
        float v[kAhead][kPer], most[kAhead];
        float to = st.m;
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            const int c = c0 + q * kWave + lane;
            u32x4 w = data[min(c, c_end - 1)];
            values(w, v[q]);
            if (c >= c_end) {
#pragma unroll
                for (int i = 0; i < kPer; ++i) v[q][i] = -INFINITY;
            }
            most[q] = v[q][0];
#pragma unroll
            for (int i = 1; i < kPer; ++i) most[q] = fmaxf(most[q], v[q][i]);
            to = fmaxf(to, most[q]);
        }
        if constexpr (TOP) {
            if (first) {
                list.bound = fmaxf(kLowest, nth_of_lanes(to, a.top));
                first = false;
            }
            // equal to the list's last at a higher place: not in it
            const bool strict = list.last != 0;
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                if (!__any(strict ? most[q] > list.bound : most[q] >= list.bound)) continue;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    if (__any(v[q][i] >= list.bound))
                        list.offer(v[q][i], head + static_cast<uint32_t>(c0 + q * kWave + lane) * kPer + i, a.top);
                }
            }
        }
        if (__any(to > st.m)) st.raise(to);
        const float at = finite_or_zero(st.m);
#pragma unroll
        for (int q = 0; q < kAhead; ++q)
#pragma unroll
            for (int i = 0; i < kPer; ++i) st.add<ENT>(v[q][i], at);
    }
    // what lies outside whole chunks: fewer than 16 values, one a lane
    if (part == 0 && wave == 0) {
        const int i = lane < head ? lane : body + lane - head;
        const bool live = lane < head || i < a.V;
        const float v = live ? logit_at<F32>(row, i) : -INFINITY;
        if constexpr (TOP) list.offer(v, i, a.top);
        st.raise(fmaxf(st.m, v));
        st.add<ENT>(v, finite_or_zero(st.m));
    }
    // lanes, then waves
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const float there[3] = {__shfl_xor(st.m, o), __shfl_xor(st.s, o), __shfl_xor(st.u, o)};
        st.join(Stats::of(there));
    }
    if (lane == 0) st.store(stats[wave]);
    if constexpr (TOP) keys[wave][lane] = lane < a.top ? list.mine : 0;
    __syncthreads();
    if (wave) return;
    for (int w = 1; w < kScoreWaves; ++w) {
        st.join(Stats::of(stats[w]));
        if constexpr (TOP) list.merge(keys[w][lane]);
    }
    if (a.parts == 1) return finish_row<F32>(a, t, row, st, list);
    const size_t at = static_cast<size_t>(t) * a.parts + part;
    if (lane == 0) st.store(a.stats + 4 * at);
    if (TOP && lane < a.top) a.keys[at * a.top + lane] = list.mine;
}

// One workgroup a row: its parts' results.
template <bool F32>
__global__ __launch_bounds__(kScoreThreads) void scores_join_kernel(ScoreArgs a, int t0) {
    __shared__ float stats[kScoreWaves][3];
    __shared__ Key keys[kScoreWaves][kWave];
    const int t = t0 + blockIdx.x;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Stats st;
    TopList list;
    for (int p = wave; p < a.parts; p += kScoreWaves) {
        const size_t at = static_cast<size_t>(t) * a.parts + p;
        st.join(Stats::of(a.stats + 4 * at));
        if (a.top) list.merge(lane < a.top ? a.keys[at * a.top + lane] : 0);
    }
    if (lane == 0) st.store(stats[wave]);
    keys[wave][lane] = list.mine;
    __syncthreads();
    if (wave) return;
    for (int w = 1; w < kScoreWaves; ++w) {
        st.join(Stats::of(stats[w]));
        list.merge(keys[w][lane]);
    }
    if (lane >= a.top) list.mine = 0;
    const char* row = static_cast<const char*>(a.logits) + t * a.stride * (F32 ? 4 : 2);
    finish_row<F32>(a, t, row, st, list);
}

template <bool F32, bool ENT, bool TOP>
hipError_t launch(const ScoreArgs& a, hipStream_t st) {
    // a grid holds fewer than 2^32 threads: rows beyond that go into further launches
    const int most = (1 << 23) / a.parts;
    for (long long t = 0; t < a.T; t += most) {
        const int n = static_cast<int>(a.T - t < most ? a.T - t : most);
        scores_kernel<F32, ENT, TOP><<<n * a.parts, kScoreThreads, 0, st>>>(a, static_cast<int>(t));
        hipError_t e = hipGetLastError();
        if (e == hipSuccess && a.parts > 1) {
            scores_join_kernel<F32><<<n, kScoreThreads, 0, st>>>(a, static_cast<int>(t));
            e = hipGetLastError();
        }
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <bool F32>
hipError_t launch_type(const ScoreArgs& a, hipStream_t st) {
    if (a.top) return a.entropy ? launch<F32, true, true>(a, st) : launch<F32, false, true>(a, st);
    return a.entropy ? launch<F32, true, false>(a, st) : launch<F32, false, false>(a, st);
}

}  // namespace

int score_parts(int T, int V) {
    int p = 1;
    while (p < 32 && static_cast<long long>(T) * p < 512 && V / (2 * p) >= 2048) p *= 2;
    return p;
}

hipError_t launch_scores(const ScoreArgs& a, bool f32, hipStream_t st) {
    return f32 ? launch_type<true>(a, st) : launch_type<false>(a, st);
}

}  // namespace qrmoe
