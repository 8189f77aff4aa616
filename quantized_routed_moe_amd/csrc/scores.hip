// Log probabilities of rows of logits (moe_token_logprobs): for every row the
// maximum m, S = sum e^(l - m), U = sum e^(l - m) (l - m) and the largest `top`
// logits in one pass; then log p = l - m - ln S, the entropy ln S - U / S.
//
// Bound by HBM with many rows (each logit is read once; 2048 x 128256 bf16, top 5, 102
// us, 5.1 TB/s of the 5.87 that reading alone reaches), by latency with few: a row is then cut into parts (1 x 128256 8.5
// us, 77 x 50001 with top 20 13, 5 x 128256 fp32 without lists 5.6).
//
// A wave takes 16 bytes a lane and chunk, four chunks a round, the next round's on
// their way; S and U are held for each lane apart, relative to the largest logit of the
// wave so far.  The wave's largest logits are a list sorted over its lanes (key:
// value, then lowest place).  A chunk whose largest value is not above the list's
// last, which is not above m, takes one comparison; else m and the list are
// looked after.  The first round would put one value after another into the list, so
// it begins with a bound: the top-th largest of the lanes' maxima, below which none of
// the row's top can be.  What is not below it, a few more than `top`, is sorted by
// counting.
//
// Logits of -inf are kept out of the lists (a masked vocabulary would fill them
// again and again): a row with fewer than `top` others takes the lowest places of
// -inf at the end.
#include <type_traits>

#include "batch.hpp"
#include "chain.hpp"
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
// The key of the lane below; lane 0 keeps its own.
__device__ __forceinline__ Key key_from_below(Key k) {
    const int lo = static_cast<int>(static_cast<uint32_t>(k)), hi = static_cast<int>(static_cast<uint32_t>(k >> 32));
    const int l = __builtin_amdgcn_update_dpp(lo, lo, 0x138, 0xf, 0xf, false);      // wave_shr:1
    const int h = __builtin_amdgcn_update_dpp(hi, hi, 0x138, 0xf, 0xf, false);
    return static_cast<Key>(static_cast<uint32_t>(h)) << 32 | static_cast<uint32_t>(l);
}

template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float dpp_max_f32(float v) {
    const int b = __float_as_int(v);
    return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(b, b, CTRL, ROW_MASK, 0xf, false)));
}
// Maximum over the 64 lanes, in every lane (the steps of wave_max_u64).
__device__ __forceinline__ float wave_max_f32(float v) {
    v = dpp_max_f32<0x111, 0xf>(v);
    v = dpp_max_f32<0x112, 0xf>(v);
    v = dpp_max_f32<0x114, 0xf>(v);
    v = dpp_max_f32<0x118, 0xf>(v);
    v = dpp_max_f32<0x142, 0xa>(v);
    v = dpp_max_f32<0x143, 0xc>(v);
    return lane_value(v, 63);
}

// A value that at least n of the lanes' are not below, and few more: the n-th
// largest of the maxima of 16, 32 or 64 groups of lanes, by counting for each those
// above it (16 take a quarter of the time of 64, and leave 6 values in the mean
// where 5 are asked for).
template <int GROUPS>
__device__ __forceinline__ float nth_of_groups(float v, int n) {
    auto flip = [](float x, auto ctrl) {
        return fmaxf(x, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), decltype(ctrl)::value, 0xf, 0xf, true)));
    };
    if constexpr (GROUPS < 64) v = flip(v, std::integral_constant<int, 0xB1>());       // lane ^ 1
    if constexpr (GROUPS < 32) v = flip(v, std::integral_constant<int, 0x4E>());       // lane ^ 2
    // the smallest value with fewer than n above it
    int above = 0;
#pragma unroll
    for (int j = 0; j < GROUPS; ++j) above += lane_value(v, j * (64 / GROUPS)) > v;
    return -wave_max_f32(above < n ? -v : -INFINITY);
}
__device__ __forceinline__ float nth_of_lanes(float v, float most, int n) {
    if (n == 1) return most;
    if (n <= 5) return nth_of_groups<16>(v, n);
    if (n <= 12) return nth_of_groups<32>(v, n);
    return nth_of_groups<64>(v, n);
}

__device__ __forceinline__ float float_below(float v) {
    const uint32_t u = __float_as_uint(v);
    return v == 0.f ? __uint_as_float(0x80000001u) : __uint_as_float(u & 0x80000000u ? u + 1 : u - 1);
}

// How many of buf's keys are above k; eight at a time, of which those from n on are
// zeros.
__device__ __forceinline__ int keys_above(const Key* buf, int n, Key k) {
    int above = 0;
    for (int j = 0; j < n; j += 8) {
        Key o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = buf[j + i];
#pragma unroll
        for (int i = 0; i < 8; ++i) above += o[i] > k;
    }
    return above;
}

// The list of a wave: lane i holds the i-th largest key of those seen.
struct TopList {
    Key mine = 0;
    Key last = 0;                              // lane top - 1's
    float bound = kLowest;                     // values below it need no look ...
    float gate = -INFINITY;                    // ... nor values not above this, at places behind the list's

    __device__ __forceinline__ void refresh(int top) {
        last = key_of_lane(mine, top - 1);
        if (last) bound = fmaxf(bound, key_value(last));
        gate = last ? bound : float_below(bound);
    }
    // Values v of the lanes (place: each lane's) that are not below the bound.
    __device__ __forceinline__ void offer(float v, uint32_t place, int top) {
        const Key k = make_key(v, place);
        const int lane = threadIdx.x & 63;
        bool in = v >= bound && k > last;
        for (uint64_t mask = __ballot(in); mask; mask = __ballot(in)) {
            const int from = __ffsll(static_cast<unsigned long long>(mask)) - 1;
            const Key n = key_of_lane(k, from);
            const int at = __popcll(__ballot(mine > n));
            const Key up = key_from_below(mine);
            mine = lane < at ? mine : lane == at ? n : up;
            refresh(top);
            in = in && k > last && lane != from;
        }
    }
    // The n <= 64 keys of buf (room for 64), sorted by counting for each those above it.
    __device__ __forceinline__ void sort(Key* buf, int n, int top) {
        const int lane = threadIdx.x & 63;
        wave_lds_fence();
        const Key k = lane < n ? buf[lane] : 0;
        if (lane >= n) buf[lane] = 0;
        wave_lds_fence();
        const int at = keys_above(buf, n, k);
        wave_lds_fence();
        if (lane < n) buf[at] = k;
        wave_lds_fence();
        mine = lane < n ? buf[lane] : 0;
        refresh(top);
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

__device__ __forceinline__ float finite_or_zero(float m) { return m == -INFINITY ? 0.f : m; }

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

template <bool F32>
__device__ __forceinline__ float logit_at(const void* row, long long i) {
    if constexpr (F32) return static_cast<const float*>(row)[i];
    else return bf16_to_f32(static_cast<const uint16_t*>(row)[i]);
}

// The first 64 given tokens of a row and their logits, asked for early: the
// lane's, or NaN.
template <bool F32>
__device__ __forceinline__ float given_logit(const ScoreArgs& a, int t, const void* row, int i) {
    if (i >= a.given) return NAN;
    const int tok = a.tokens[static_cast<size_t>(t) * a.given + i];
    const float l = logit_at<F32>(row, min(max(tok, 0), a.V - 1));
    return tok >= 0 && tok < a.V ? l : NAN;
}

// Outputs of row t from its statistics and the lanes' keys, by one wave.
template <bool F32>
__device__ __forceinline__ void finish_row(const ScoreArgs& a, int t, const void* row, const Stats& st, Key mine, float given) {
    const int lane = threadIdx.x & 63;
    const float m = finite_or_zero(st.m), ln_s = logf(st.s);      // all -inf: m 0, ln 0 = -inf; NaN if a logit was NaN or +inf
    const bool empty = st.s == 0.f, bad = st.s != st.s;
    auto logprob = [&](float l) { return bad || l != l ? NAN : empty ? -INFINITY : (l - m) - ln_s; };
    if (a.entropy && lane == 0) a.entropy[t] = empty ? 0.f : ln_s - st.u / st.s;
    for (int i = lane; i < a.given; i += 64)
        a.logprobs[static_cast<size_t>(t) * a.given + i] = logprob(i < 64 ? given : given_logit<F32>(a, t, row, i));
    if (!a.top) return;
    // places of -inf in order, if the others do not fill the list: they are
    // fewer than top, so the first 128 places hold enough
    int found = __popcll(__ballot(mine != 0));
    for (int i0 = 0; !bad && found < a.top && i0 < a.V; i0 += 64) {
        const int i = i0 + lane;
        const uint64_t hidden = __ballot(i < a.V && logit_at<F32>(row, min(i, a.V - 1)) == -INFINITY);
        const int here = __popcll(hidden);
        // lane found + j takes the j-th
        uint64_t left = hidden;
        for (int j = 0; j < here && found + j < a.top; ++j, left &= left - 1)
            if (lane == found + j) mine = make_key(-INFINITY, i0 + __ffsll(static_cast<unsigned long long>(left)) - 1);
        found += here;
    }
    if (lane < a.top) {
        const size_t at = static_cast<size_t>(t) * a.top + lane;
        const bool none = bad || !mine;
        a.top_ids[at] = none ? -1 : static_cast<int>(key_place(mine));
        a.top_logprobs[at] = none ? NAN : logprob(key_value(mine));
    }
}

// A row in memory: values before the first whole 16 bytes, whole chunks, values
// after them.
template <bool F32>
struct Row {
    static constexpr int per = F32 ? 4 : 8;    // values of a chunk
    const char* p;
    const u32x4* data;
    int head, chunks, V;
    __device__ __forceinline__ Row(const ScoreArgs& a, int t) {
        constexpr int kBytes = F32 ? 4 : 2;
        p = static_cast<const char*>(a.logits) + t * a.stride * kBytes;
        V = a.V;
        head = min(static_cast<int>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / kBytes, V);
        chunks = (V - head) / per;
        data = reinterpret_cast<const u32x4*>(p + head * kBytes);
    }
    // Values of the chunks from c on, one a lane, `past` if there is none.
    static __device__ __forceinline__ void values(u32x4 raw, int c, int c_end, float (&v)[per]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = raw[i];
            if constexpr (F32) {
                v[i] = __uint_as_float(w);
            } else {
                v[2 * i] = bf16lo(w);
                v[2 * i + 1] = bf16hi(w);
            }
        }
        if (c + kWave > c_end) {
            const bool past = c + static_cast<int>(threadIdx.x & 63) >= c_end;
#pragma unroll
            for (int i = 0; i < per; ++i) v[i] = past ? -INFINITY : v[i];
        }
    }
    static __device__ __forceinline__ float largest(const float (&v)[per]) {
        float m = v[0];
#pragma unroll
        for (int i = 1; i < per; ++i) m = fmaxf(m, v[i]);
        return m;
    }
    __device__ __forceinline__ uint32_t place(int c, int i) const {
        return head + static_cast<uint32_t>(c + (threadIdx.x & 63)) * per + i;
    }
    // What lies outside whole chunks, fewer than 16 values, one a lane; -inf past them.
    __device__ __forceinline__ int edge_place() const {
        const int lane = threadIdx.x & 63;
        return lane < head ? lane : chunks * per + lane;
    }
    __device__ __forceinline__ bool has_edge() const { return head || head + chunks * per < V; }
    __device__ __forceinline__ float edge() const {
        const int i = edge_place();
        const float v = logit_at<F32>(p, min(i, V - 1));
        return i < V ? v : -INFINITY;
    }
};

// A wave's share of a row: of its chunks [c_beg, c_end), 64 at a time, every
// WAVES-th from `first` on, and, if edges, what lies outside whole chunks.
template <bool F32, bool ENT, bool TOP, int WAVES>
__device__ __forceinline__ void wave_share(const ScoreArgs& a, const Row<F32>& row, int c_beg, int c_end, int first, bool edges,
                                           Key* buf, Stats& st, TopList& list) {
    constexpr int kPer = Row<F32>::per, kChunks = WAVES == 1 ? 8 : 4;
    constexpr int kApart = WAVES * kWave, kRound = kChunks * kApart;
    const int lane = threadIdx.x & 63;
    u32x4 raw[kChunks], next[kChunks];
    // read once: past the caches (2048 x 128256 112 -> 104 us)
    auto load = [&](int c0, u32x4 (&to)[kChunks]) {
#pragma unroll
        for (int q = 0; q < kChunks; ++q) to[q] = __builtin_nontemporal_load(row.data + min(c0 + q * kApart + lane, c_end - 1));
    };
    auto values = [&](int c0, int q, float (&v)[kPer]) { row.values(raw[q], c0 + q * kApart, c_end, v); };
    auto largest = [&](const float (&v)[kPer]) { return row.largest(v); };
    auto place = [&](int c0, int q, int i) { return row.place(c0 + q * kApart, i); };

    int c0 = c_beg + first * kWave;
    bool fresh = true;                         // m and the list have not begun
    if (c0 < c_end) load(c0, raw);
    while (c0 < c_end) {
        const int c1 = c0 + kRound;
        if (c1 < c_end) load(c1, next);
        bool listed = false;                   // this round's values are in the list already
        if (fresh) {
            fresh = false;
            float most = -INFINITY, v[kPer];
#pragma unroll
            for (int q = 0; q < kChunks; ++q) {
                if (c0 + q * kApart >= c_end) break;
                values(c0, q, v);
                most = fmaxf(most, largest(v));
            }
            st.m = wave_max_f32(most);
            if constexpr (TOP) {
                list.bound = fmaxf(kLowest, nth_of_lanes(most, st.m, a.top));
                int n = 0;
#pragma unroll
                for (int q = 0; q < kChunks; ++q) {
                    if (c0 + q * kApart >= c_end) break;
                    values(c0, q, v);
                    if (!__any(largest(v) >= list.bound)) continue;
#pragma unroll
                    for (int i = 0; i < kPer; ++i) {
                        const bool in = v[i] >= list.bound;
                        const uint64_t mask = __ballot(in);
                        if (!mask) continue;
                        const int at = n + __popcll(mask & (lane ? ~0ull >> (64 - lane) : 0ull));
                        if (in && at < kWave) buf[at] = make_key(v[i], place(c0, q, i));
                        n += __popcll(mask);
                    }
                }
                listed = n <= kWave;
                if (listed) list.sort(buf, n, a.top);
                else list.refresh(a.top);
            }
        }
#pragma unroll
        for (int q = 0; q < kChunks; ++q) {
            if (c0 + q * kApart >= c_end) break;
            float v[kPer];
            values(c0, q, v);
            const float most = largest(v);
            if (!listed && __any(most > (TOP ? list.gate : st.m))) {
                if (__any(most > st.m)) st.raise(wave_max_f32(fmaxf(most, st.m)));
                if constexpr (TOP) {
#pragma unroll
                    for (int i = 0; i < kPer; ++i)
                        if (__any(v[i] >= list.bound)) list.offer(v[i], place(c0, q, i), a.top);
                }
            }
            const float at = finite_or_zero(st.m);
#pragma unroll
            for (int i = 0; i < kPer; ++i) st.add<ENT>(v[i], at);
        }
        c0 = c1;
#pragma unroll
        for (int q = 0; q < kChunks; ++q) raw[q] = next[q];
    }
    if (edges) {
        const float v = row.edge();
        if constexpr (TOP) list.offer(v, row.edge_place(), a.top);
        st.raise(wave_max_f32(fmaxf(st.m, v)));
        st.add<ENT>(v, finite_or_zero(st.m));
    }
    st.s = wave_sum_f32(st.s);
    st.u = wave_sum_f32(st.u);
}

__device__ __forceinline__ void store_device(float* p, float v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float load_device(const float* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ Key load_device(const Key* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

constexpr int kBuf = kScoreThreads;            // keys that a workgroup sorts by counting

struct Shared {
    Key buf[kBuf];
    Key keys[kScoreWaves][kWave];
    Key merged[kWave];
    float groups[128];
    float stats[kScoreWaves][3];
    int count;
};

// sh.merged from the sh.count <= kBuf keys of sh.buf (zeros behind them).
__device__ __forceinline__ void sort_buf(Shared& sh, int top) {
    const int count = sh.count;
    if (static_cast<int>(threadIdx.x) < count) {
        const Key k = sh.buf[threadIdx.x];
        const int at = keys_above(sh.buf, count, k);
        if (k && at < top) sh.merged[at] = k;
    }
}

// sh.merged from the waves' lists.
__device__ __forceinline__ void merge_waves(Shared& sh, const TopList& list, int top) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const bool in = lane < top;
    sh.buf[in ? wave * top + lane : kScoreWaves * top + wave * (kWave - top) + lane - top] = in ? list.mine : 0;
    if (threadIdx.x == 0) sh.count = kScoreWaves * top;
    __syncthreads();
    sort_buf(sh, top);
    __syncthreads();
}

__device__ __forceinline__ void append(Shared& sh, Key k) {
    const int at = atomicAdd(&sh.count, 1);
    if (at < kBuf) sh.buf[at] = k;
}

// One workgroup: row t from its parts' results.  Of the parts' sorted lists, the
// keys that can be among the top are not below the q-th largest of their j-th, q j >= top.
template <bool F32>
__device__ __forceinline__ void join_row(const ScoreArgs& a, int t, const char* row, float given, Shared& sh) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const size_t slot = static_cast<size_t>(t) * a.parts;
    const float* from_st = a.stats + 4 * (slot + min(lane, a.parts - 1));
    Stats st;
    st.m = load_device(from_st);
    st.s = load_device(from_st + 1);
    st.u = load_device(from_st + 2);
    Key mine = 0;
    if (a.top) {
        const Key* from = a.keys + slot * a.top;
        const int j = (a.top + a.parts - 1) / a.parts, q = (a.top + j - 1) / j, n = a.parts * a.top;
        const Key k = lane < a.parts ? load_device(from + lane * a.top + j - 1) : 0;
        const Key first = static_cast<int>(threadIdx.x) < n ? load_device(from + threadIdx.x) : 0;
        sh.keys[wave][lane] = k;               // each wave for itself
        sh.buf[threadIdx.x] = 0;
        if (wave == 0) sh.merged[lane] = 0;
        if (threadIdx.x == 0) sh.count = 0;
        wave_lds_fence();
        const int above = keys_above(sh.keys[wave], a.parts, k);               // places differ: only zeros are equal
        const uint64_t hit = __ballot(above == q - 1 && k);
        const Key least = hit ? key_of_lane(k, __ffsll(static_cast<unsigned long long>(hit)) - 1) : 1;
        __syncthreads();
        if (first >= least) append(sh, first);
        for (int i = threadIdx.x + kScoreThreads; i < n; i += kScoreThreads) {
            const Key c = load_device(from + i);
            if (c >= least) append(sh, c);
        }
        __syncthreads();
        if (sh.count <= kBuf) {
            sort_buf(sh, a.top);
            __syncthreads();
            mine = sh.merged[lane];
        } else {                               // many lists that lie within one another
            __syncthreads();                   // sh.count is read by all
            TopList list;
            for (int p = wave; p < a.parts; p += kScoreWaves) list.merge(lane < a.top ? load_device(from + p * a.top + lane) : 0);
            merge_waves(sh, list, a.top);
            mine = sh.merged[lane];
        }
    }
    if (wave) return;
    if (lane >= a.parts) st = Stats();
    st.raise(wave_max_f32(st.m));
    st.s = wave_sum_f32(st.s);
    st.u = wave_sum_f32(st.u);
    finish_row<F32>(a, t, row, st, mine, given);
}

// A workgroup's chunks of a row, seen twice: first the maxima of groups of lanes,
// from which follow m and a bound that at least `top` values are not below; then the sums
// relative to m, and the values not below the bound, a few more than `top`, into
// sh.buf.  Up to 4 chunks a lane stay in registers in between, more are read again.
// Leaves the wave's S and U, and sh.merged.
template <bool F32, bool ENT, bool TOP>
__device__ __forceinline__ void share_twice(const ScoreArgs& a, const Row<F32>& row, int c_beg, int c_end, bool edges, Shared& sh,
                                            Stats& st) {
    constexpr int kPer = Row<F32>::per, kChunks = 4, kRound = kChunks * kScoreThreads;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int first = c_beg + wave * kWave;
    u32x4 raw[kChunks];
    auto load = [&](int c0) {
#pragma unroll
        for (int q = 0; q < kChunks; ++q) raw[q] = row.data[min(c0 + q * kScoreThreads + lane, c_end - 1)];
    };
    const float edge = edges ? row.edge() : -INFINITY;
    float most = edge;
    const bool once = c_end - c_beg <= kRound;
    for (int c0 = first; c0 < c_end; c0 += kRound) {
        load(c0);
#pragma unroll
        for (int q = 0; q < kChunks; ++q) {
            if (c0 + q * kScoreThreads >= c_end) break;
            float v[kPer];
            row.values(raw[q], c0 + q * kScoreThreads, c_end, v);
            most = fmaxf(most, row.largest(v));
        }
    }
    // groups of 64 / per lanes: about three times `top` of them or more
    const int per = !TOP || a.top <= 5 ? 4 : a.top <= 10 ? 8 : a.top <= 21 ? 16 : 32, G = kScoreWaves * per;
    auto flip = [&](auto ctrl) {
        most = fmaxf(most, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(most), decltype(ctrl)::value, 0xf, 0xf, true)));
    };
    flip(std::integral_constant<int, 0xB1>());                 // 2 lanes
    if (per <= 16) flip(std::integral_constant<int, 0x4E>());  // 4
    if (per <= 8) flip(std::integral_constant<int, 0x141>());  // 8: row_half_mirror
    if (per <= 4) flip(std::integral_constant<int, 0x140>());  // 16: row_mirror
    if (lane % (kWave / per) == 0) sh.groups[wave * per + lane / (kWave / per)] = most;
    if constexpr (TOP) {
        sh.buf[threadIdx.x] = 0;
        if (wave == 0) sh.merged[lane] = 0;
        if (threadIdx.x == 0) sh.count = 0;
    }
    __syncthreads();
    const float g0 = lane < G ? sh.groups[lane] : -INFINITY, g1 = G > kWave ? sh.groups[kWave + lane] : -INFINITY;
    st.m = wave_max_f32(fmaxf(g0, g1));
    float bound = INFINITY;
    if constexpr (TOP) {
        // the smallest with fewer than top above it
        int above0 = 0, above1 = 0;
        for (int j = 0; j < G; j += 8) {
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = sh.groups[j + i];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                above0 += o[i] > g0;
                above1 += o[i] > g1;
            }
        }
        bound = fmaxf(kLowest, -wave_max_f32(fmaxf(lane < G && above0 < a.top ? -g0 : -INFINITY,
                                                   G > kWave && above1 < a.top ? -g1 : -INFINITY)));
    }
    const float at = finite_or_zero(st.m);
    for (int c0 = first; c0 < c_end; c0 += kRound) {
        if (!once) load(c0);
#pragma unroll
        for (int q = 0; q < kChunks; ++q) {
            const int c = c0 + q * kScoreThreads;
            if (c >= c_end) break;
            float v[kPer];
            row.values(raw[q], c, c_end, v);
#pragma unroll
            for (int i = 0; i < kPer; ++i) st.add<ENT>(v[i], at);
            if constexpr (TOP) {
                if (!__any(row.largest(v) >= bound)) continue;
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (v[i] >= bound) append(sh, make_key(v[i], row.place(c, i)));
            }
        }
    }
    if (edges) {
        st.add<ENT>(edge, at);
        if (TOP && edge >= bound) append(sh, make_key(edge, row.edge_place()));
    }
    st.s = wave_sum_f32(st.s);
    st.u = wave_sum_f32(st.u);
    if constexpr (TOP) {
        __syncthreads();
        if (sh.count <= kBuf) {
            sort_buf(sh, a.top);
            __syncthreads();
        } else {                               // many equal to the bound: one after the other
            __syncthreads();                   // sh.count is read by all
            Stats again;
            TopList list;
            wave_share<F32, false, true, kScoreWaves>(a, row, c_beg, c_end, wave, edges, sh.keys[wave], again, list);
            merge_waves(sh, list, a.top);
        }
    }
}

// What a workgroup takes: a row of each wave; a row, seen once; a row or a part of
// one, seen twice.  The parts of a row are joined by the workgroup that finds them
// all there: each stores its results, raises its flag (a value unique to the launch, see
// chain.hpp, so nothing has to be cleared) once they are acknowledged, and reads the
// row's flags once that is acknowledged too: whichever is last sees them all.  When
// several do, they store the same bytes.  Nobody waits for another.
template <bool F32, bool ENT, bool TOP, ScoreTake TAKE>
__global__ __launch_bounds__(kScoreThreads, TAKE == ScoreTake::kRows ? 4 : 5) void scores_kernel(ScoreArgs a, int t0, int n) {
    constexpr bool ROWS = TAKE == ScoreTake::kRows, PART = TAKE == ScoreTake::kPart;
    __shared__ Shared sh;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int at = ROWS ? blockIdx.x * kScoreWaves + wave : PART ? blockIdx.x / a.parts : blockIdx.x;
    const int part = PART ? blockIdx.x % a.parts : 0, parts = PART ? a.parts : 1;
    if (ROWS && at >= n) return;
    const int t = t0 + at;
    const Row<F32> row(a, t);
    const float given = ROWS || wave == 0 ? given_logit<F32>(a, t, row.p, lane) : NAN;
    Stats st;
    if constexpr (TAKE == ScoreTake::kRows) {
        TopList list;
        wave_share<F32, ENT, TOP, 1>(a, row, 0, row.chunks, 0, row.has_edge(), sh.keys[wave], st, list);
        return finish_row<F32>(a, t, row.p, st, lane < a.top ? list.mine : 0, given);
    } else if constexpr (TAKE == ScoreTake::kRow) {
        TopList list;
        wave_share<F32, ENT, TOP, kScoreWaves>(a, row, 0, row.chunks, wave, wave == 0 && row.has_edge(), sh.keys[wave], st, list);
        if (lane == 0) st.store(sh.stats[wave]);
        if (TOP && wave == 0) sh.merged[lane] = 0;
        __syncthreads();
        if constexpr (TOP) merge_waves(sh, list, a.top);
    } else {
        const int c_beg = static_cast<int>(static_cast<long long>(row.chunks) * part / parts);
        const int c_end = static_cast<int>(static_cast<long long>(row.chunks) * (part + 1) / parts);
        share_twice<F32, ENT, TOP>(a, row, c_beg, c_end, part == 0 && wave == 0 && row.has_edge(), sh, st);
        if (lane == 0) st.store(sh.stats[wave]);
        __syncthreads();
    }
    if (wave == 0)
        for (int w = 1; w < kScoreWaves; ++w) st.join(Stats::of(sh.stats[w]));
    if (parts == 1) {
        if (wave == 0) finish_row<F32>(a, t, row.p, st, TOP ? sh.merged[lane] : 0, given);
        return;
    }
    if constexpr (PART) {
        const size_t slot = static_cast<size_t>(t) * a.parts;
        const unsigned long long tag = chain_tag();
        if (wave == 0) {
            if (lane < 3) store_device(a.stats + 4 * (slot + part) + lane, lane == 0 ? st.m : lane == 1 ? st.s : st.u);
            if (TOP && lane < a.top)
                __hip_atomic_store(a.keys + (slot + part) * a.top + lane, sh.merged[lane], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        raise_flag(a.flags + slot + part, tag);
        if (wave == 0) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            const bool there = lane >= a.parts || load_device(a.flags + slot + lane) == tag;
            const bool all = __all(there);
            if (lane == 0) sh.count = all;
        }
        __syncthreads();
        const int all = sh.count;
        __syncthreads();
        if (all) join_row<F32>(a, t, row.p, given, sh);
    }
}

template <bool F32, bool ENT, bool TOP>
hipError_t launch(const ScoreArgs& a, hipStream_t st) {
    // a grid holds fewer than 2^32 threads: rows beyond that go into further launches
    const int most = (1 << 23) / a.parts;
    for (long long t = 0; t < a.T; t += most) {
        const int n = static_cast<int>(a.T - t < most ? a.T - t : most), first = static_cast<int>(t);
        if (a.take == ScoreTake::kPart) scores_kernel<F32, ENT, TOP, ScoreTake::kPart><<<n * a.parts, kScoreThreads, 0, st>>>(a, first, n);
        else if (a.take == ScoreTake::kRow) scores_kernel<F32, ENT, TOP, ScoreTake::kRow><<<n, kScoreThreads, 0, st>>>(a, first, n);
        else scores_kernel<F32, ENT, TOP, ScoreTake::kRows><<<ceil_div(n, kScoreWaves), kScoreThreads, 0, st>>>(a, first, n);
        const hipError_t e = hipGetLastError();
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

// Parts of a row: as many as make about a thousand workgroups, of 2000 values or
// more (us, top 5 of bf16: 1 x 128256 in 8 / 16 / 32 parts 9.9 / 8.7 / 8.5; 16 x 32000
// in 8 / 16 / 32 8.2 / 7.9 / 8.9; 300 x 32000 in 1 / 2 / 4 / 8 16.7 / 14.9 / 14.1 / 19.0);
// beyond a thousand, of 6000 (77 x 50001, top 20, in 8 / 16 12.9 / 15.1; 77 x
// 128256 14.8 / 13.9).  A row of 16 KB is not worth the join (16 x 8192 in 1 / 2 6.2 /
// 8.1, 16 x 16384 9.4 / 8.7).
int score_parts(int T, int V, bool f32) {
    if (static_cast<long long>(V) * (f32 ? 4 : 2) <= 16384) return 1;
    int p = 1;
    while (p < 32) {
        const int n = 2 * p;
        const long long blocks = static_cast<long long>(T) * n;
        if (blocks > 1240 || V / n < (blocks <= 1024 ? 2000 : 6000)) break;
        p = n;
    }
    return p;
}

// Whole rows (us, bf16): a row a wave where there are waves enough and little to
// do in each (top 5: 4096 x 1000 7.5, a row a workgroup 13.3; 2048 x 4096 9.9, 11.9;
// 2048 x 8192 17.4, 14.9; 512 x 4096 7.1, 6.0); seen twice for long lists of rows up
// to 32 KB (1024 x 16384: top 20 17.6, once 23.4, top 5 15.1, 16.6, none 12.2, 10.5;
// 512 x 8192 8.7, 9.2; 7.0, 7.0; 4.8, 4.3; 2048 x 32000, top 5, 45.7, 40.8).
ScoreTake score_take(int T, int V, int top, bool f32, int parts) {
    const long long bytes = static_cast<long long>(V) * (f32 ? 4 : 2);
    if (parts > 1) return ScoreTake::kPart;
    if (T >= 2048 && bytes <= 8192) return ScoreTake::kRows;
    return top > 5 && bytes <= 32768 ? ScoreTake::kPart : ScoreTake::kRow;
}

hipError_t launch_scores(const ScoreArgs& a, bool f32, hipStream_t st) {
    return f32 ? launch_type<true>(a, st) : launch_type<false>(a, st);
}

}  // namespace qrmoe
