// Low-rank adapters of many requests beside a shared projection (moe_lora_add):
// v = a[g] x for every token with an adapter g, then out = base + scales[g] b[g] v.
//
// Few operations a byte: bound by HBM (x, the active adapters, base and out),
// with few tokens by the launch and a chain of latencies.  One launch.  First come
// the workgroups that make v: a run of up to 32 tokens of one adapter, up to 32
// ranks and a part of K, which their waves split, their sums meeting in LDS in wave
// order.  Then those of the columns: up to 32 tokens of a run x 512 columns, whose
// weights and base are on their way while they wait for v by its flags; they add
// its parts in order, so nothing depends on timing.  One that has waited long makes
// its tokens' v itself.  (In two launches 2048 tokens x 4096 x 4096 at rank 32 took
// 21.2 us, in one 16.8; 64 tokens of 64 adapters at rank 16 10.2 and 8.2.)
//
// Both are 16x16x32 bf16 products, exact in fp32 but for the sums.  v is fp32: for
// the columns it is split into three bf16 parts that hold its 24 bits, and three
// products are added (the matrix work is a few per cent of the time that base and
// out take).
//
// A load whose neighbouring lanes are in different rows takes 3.4 times as long as
// one whose four lanes of a quad share 64 bytes (128 KB by one workgroup: 3.4 and
// 1.0 us).  So x and a are loaded as lane = (row, 16-byte chunk) and turned into the
// instruction's (chunk, row) by lane exchanges, b goes through LDS, and the product
// of the columns has tokens as operand A and, as column c of fragment f, weight row
// 8 c + f, so that a lane's eight fragments are eight neighbouring columns of its
// four tokens.
//
// Up to four tokens: few_body.
#include "batch.hpp"
#include "chain.hpp"

namespace qrmoe {

namespace {

constexpr int kWaves = 4;                      // of a workgroup that makes v or columns
constexpr int kCols = 128 * kWaves;
constexpr int kHalfRows = 32, kHalves = kItemRows / kHalfRows;
constexpr int kStep = 128;                     // values of K of four products
constexpr int kMostSplits = 8;
constexpr int kFewWaves = 8;
constexpr int kFewCols = 2 * kFewWaves * kWave;

struct Run {
    int g, r0, r1;
};

// Item i of the plan, its bounds made sound; g < 0: nothing to do.
__device__ __forceinline__ Run load_run(const LoraArgs& a, int i) {
    const int4 v = reinterpret_cast<const int4*>(a.items)[i];
    Run r{__builtin_amdgcn_readfirstlane(v.x), __builtin_amdgcn_readfirstlane(v.y), __builtin_amdgcn_readfirstlane(v.z)};
    r.r0 = max(r.r0, 0);
    r.r1 = min(min(r.r1, a.T), r.r0 + kItemRows);
    if (r.g < 0 || r.g > a.L || r.r0 >= r.r1) r.g = -1;
    return r;
}

// No load before this point is moved behind it: left to itself the compiler puts
// each load into the branch that uses it and waits there.
__device__ __forceinline__ void hold_loads() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Four loads of a lane as four operands: load i holds chunk l % 4 (16 bytes) of
// piece l / 16 of row 4 (l / 4 % 4) + i; operand i is to hold chunk i of piece
// l / 16 of row l % 16, which is a transposition within every four lanes.
__device__ __forceinline__ void turn(const u32x4 (&v)[4], bf16x8 (&o)[4]) {
    const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
    auto flip1 = [](uint32_t x) { return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0xB1, 0xf, 0xf, true)); };
    auto flip2 = [](uint32_t x) { return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x4E, 0xf, 0xf, true)); };
    u32x4 r[4];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        uint32_t a[4];
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const uint32_t even = flip1(v[i][d]), next = flip1(v[i + 1][d]);       // by all lanes
            a[i] = odd ? next : v[i][d];
            a[i + 1] = odd ? v[i + 1][d] : even;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t low = flip2(a[i]), next = flip2(a[i + 2]);
            r[i][d] = high ? next : a[i];
            r[i + 2][d] = high ? a[i + 2] : low;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = bf16x8_from_u32x4(r[i]);
}

// Sums of a wave's steps [beg, end) of K: ranks j0 + 16 f + .. times the run's
// tokens 16 q + ..; lane l has ranks 4 (l / 16) + i of token l % 16.  AHEAD: steps
// on their way.
template <int RF, int TT, int AHEAD>
struct Sums {
    f32x4 acc[RF * TT];
    u32x4 av[AHEAD][RF][4], xv[AHEAD][TT][4];
    const uint16_t *arow, *xrow[TT][4];        // arow: of fragment 0 (uniform)
    int aoff[RF];                              // the lane's place in a fragment

    static __device__ __forceinline__ int lane_k() { return 8 * (threadIdx.x & 3) + 32 * (threadIdx.x >> 4 & 3); }

    // Rows, and the first steps' loads.
    __device__ __forceinline__ void begin(const LoraArgs& a, const Run& run, int j0, int beg, int end) {
        const int row = a.tid & 12;
        int t[TT][4];
#pragma unroll
        for (int q = 0; q < TT; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) t[q][i] = a.perm[min(run.r0 + 16 * q + row + i, run.r1 - 1)];
        arow = a.a + (static_cast<size_t>(run.g) * a.r + j0) * a.K;
#pragma unroll
        for (int f = 0; f < RF; ++f) aoff[f] = min(16 * f + row, a.r - j0 - 4) * a.K;      // r is a multiple of 8
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) load_a(a, u, beg + u, end);
#pragma unroll
        for (int q = 0; q < TT; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) xrow[q][i] = a.x + (t[q][i] >= 0 && t[q][i] < a.T ? t[q][i] : 0) * a.x_stride;
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
#pragma unroll
            for (int q = 0; q < TT; ++q) load_x(a, u, q, beg + u, end);
#pragma unroll
        for (int i = 0; i < RF * TT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    // The lane's place in step s; past K (a multiple of 32) or the last step any other.
    static __device__ __forceinline__ int place(const LoraArgs& a, int s, int end) {
        const int k = kStep * min(s, max(end - 1, 0)) + lane_k();
        return k < a.K ? k : lane_k() < a.K ? lane_k() : 0;
    }
    __device__ __forceinline__ void load_a(const LoraArgs& a, int u, int s, int end) {
        const int k = place(a, s, end);
#pragma unroll
        for (int f = 0; f < RF; ++f)
#pragma unroll
            for (int i = 0; i < 4; ++i) av[u][f][i] = *reinterpret_cast<const u32x4*>(arow + i * a.K + (aoff[f] + k));
    }
    __device__ __forceinline__ void load_x(const LoraArgs& a, int u, int q, int s, int end) {
        const int k = place(a, s, end);
#pragma unroll
        for (int i = 0; i < 4; ++i) xv[u][q][i] = *reinterpret_cast<const u32x4*>(xrow[q][i] + k);
    }
    // Step s, held in slot u; NEXT: each operand's place is asked to hold step s + AHEAD
    // as soon as it is free.
    template <bool NEXT>
    __device__ __forceinline__ void step(const LoraArgs& a, int u, int s, int end) {
        if (kStep * (s + 1) > a.K && kStep * s + lane_k() >= a.K) {
#pragma unroll
            for (int q = 0; q < TT; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) xv[u][q][i] = u32x4{0u, 0u, 0u, 0u};
        }
        bf16x8 ao[RF][4];
#pragma unroll
        for (int f = 0; f < RF; ++f) turn(av[u][f], ao[f]);
        if constexpr (NEXT) {
            load_a(a, u, s + AHEAD, end);
            hold_loads();
        }
#pragma unroll
        for (int q = 0; q < TT; ++q) {
            bf16x8 xo[4];
            turn(xv[u][q], xo);
            if constexpr (NEXT) {
                load_x(a, u, q, s + AHEAD, end);
                hold_loads();
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int f = 0; f < RF; ++f) acc[f * TT + q] = mfma16x16x32(ao[f][i], xo[i], acc[f * TT + q]);
        }
    }
    __device__ __forceinline__ void run_steps(const LoraArgs& a, int beg, int end) {
        hold_loads();
        int s = beg;
        for (; s + 2 * AHEAD <= end; s += AHEAD)
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) step<true>(a, u, s + u, end);
        for (; s < end; s += AHEAD) {
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                if (s + u >= end) break;
                step<false>(a, u, s + u, end);
            }
            if (AHEAD > 1 && s + AHEAD < end) {
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) {
                    load_a(a, u, s + AHEAD + u, end);
#pragma unroll
                    for (int q = 0; q < TT; ++q) load_x(a, u, q, s + AHEAD + u, end);
                }
                hold_loads();
            }
        }
    }
};

// The rows of v of a run and part of K, for accesses that other workgroups of the launch
// see and whose whole 16 bytes count as one.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t v_rows(const LoraArgs& a, const Run& run, int split) {
    return __builtin_amdgcn_make_buffer_rsrc(a.v + (static_cast<size_t>(split) * a.T + run.r0) * a.r, 0, kHalfRows * a.r * 4, 4 << 15);
}

// The workgroup's part `split` of K and ranks from j0 on.  The waves' sums are
// added in wave order; v is read by other workgroups of this launch.
template <int RF, int TT>
__device__ __forceinline__ void make_v(const LoraArgs& a, const Run& run, int split, int j0, f32x4* part) {
    const int lane = a.tid & 63, wave = __builtin_amdgcn_readfirstlane(a.tid >> 6);
    const long long steps = ceil_div(a.K, kStep);
    const int slice = split * kWaves + wave, slices = a.splits * kWaves;
    const int beg = steps * slice / slices, end = steps * (slice + 1) / slices;
    Sums<RF, TT, (RF + TT <= 2 ? 2 : 1)> sums;
    sums.begin(a, run, j0, beg, end);
    sums.run_steps(a, beg, end);
    const auto to = v_rows(a, run, split);
#pragma unroll
    for (int i = 0; i < RF * TT; ++i) part[(wave * RF * TT + i) * kWave + lane] = sums.acc[i];
    __syncthreads();
    // four ranks of a token, neighbouring threads in a row; r is a multiple of 8
    for (int i = a.tid; i < RF * TT * kWave; i += kWaves * kWave) {
        const int row = i / (4 * RF), quad = i % (4 * RF), j = j0 + 4 * quad;
        const int from = (quad / 4 * TT + row / 16) * kWave + 16 * (quad % 4) + row % 16;
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) s += part[w * RF * TT * kWave + from];
        if (run.r0 + row < run.r1 && j < a.r)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, s), to, (row * a.r + j) * 4, 0, kAuxDevice);
    }
}

// Up to 32 tokens of an item: the first halves of all items, then the second,
// of which few have tokens where adapters have few: workgroups go round the XCDs,
// and alternating halves left every second XCD idle.
__device__ __forceinline__ Run load_half(const LoraArgs& a, int at) {
    Run run = load_run(a, at % a.n_items);
    run.r0 += kHalfRows * (at / a.n_items);
    run.r1 = min(run.r1, run.r0 + kHalfRows);
    if (run.r0 >= run.r1) run.g = -1;
    return run;
}

// Two floats to bf16, nearest even, in one instruction (a NaN stays one).
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// Three bf16 parts of four floats, exact to 2^-24: each subtraction is exact
// and each part takes the next 8 bits.
__device__ __forceinline__ void split_parts(const f32x4& v, u32x2 (&p)[3]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float a = v[2 * i], b = v[2 * i + 1];
#pragma unroll
        for (int q = 0; q < 3; ++q) {
            p[q][i] = bf16_pair(a, b);
            a -= bf16lo(p[q][i]);
            b -= bf16hi(p[q][i]);
        }
    }
}

// A lane's eight values of a row of base or out.  VEC: eight neighbouring
// columns from n on, whole 16 bytes, N a multiple of 8.  Else values 16 columns apart,
// so that neighbouring lanes have neighbouring columns.  Loads are unconditional
// (n is clamped) and converted when they are used.
template <bool F32, bool VEC>
struct Eight {
    static constexpr int step = VEC ? 1 : 16;
    static constexpr int words = VEC ? (F32 ? 8 : 4) : 8;
    uint32_t w[words];
    __device__ __forceinline__ void load(const void* base, long long row, int n, int N) {
        if constexpr (VEC) {
            const char* p = static_cast<const char*>(base) + (row + min(n, N - 8)) * (F32 ? 4 : 2);
#pragma unroll
            for (int h = 0; h < words / 4; ++h) {
                const u32x4 v = reinterpret_cast<const u32x4*>(p)[h];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[4 * h + i] = v[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const long long at = row + min(n + step * i, N - 1);
                w[i] = F32 ? static_cast<const uint32_t*>(base)[at] : static_cast<const uint16_t*>(base)[at];
            }
        }
    }
    __device__ __forceinline__ float value(int i) const {
        if constexpr (F32) return __uint_as_float(w[i]);
        else if constexpr (VEC) return i % 2 ? bf16hi(w[i / 2]) : bf16lo(w[i / 2]);
        else return bf16lo(w[i]);
    }
};

template <bool F32, bool VEC>
__device__ __forceinline__ void store8(void* out, long long row, int n, int N, const float (&v)[8]) {
    if constexpr (VEC) {
        if (n >= N) return;
        char* p = static_cast<char*>(out) + (row + n) * (F32 ? 4 : 2);
        if constexpr (F32) {
            reinterpret_cast<f32x4*>(p)[0] = f32x4{v[0], v[1], v[2], v[3]};
            reinterpret_cast<f32x4*>(p)[1] = f32x4{v[4], v[5], v[6], v[7]};
        } else {
            u32x4 w;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
            *reinterpret_cast<u32x4*>(p) = w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (n + 16 * i >= N) break;
            if constexpr (F32) static_cast<float*>(out)[row + n + 16 * i] = v[i];
            else static_cast<uint16_t*>(out)[row + n + 16 * i] = static_cast<uint16_t>(bf16_pair(v[i], v[i]));
        }
    }
}

// The tokens' v as operands: three parts of ROWS rows of ranks, a row's 32 KS
// ranks and 16 bytes more, so that 16 rows' chunks lie in distinct banks.
template <int ROWS, int KS>
struct Parts {
    static constexpr int row_bytes = 64 * KS + 16;
    uint8_t b[3][ROWS][row_bytes];
    // ranks j .. j + 3 of a row
    __device__ __forceinline__ void set(int row, int j, const f32x4& v) {
        u32x2 p[3];
        split_parts(v, p);
#pragma unroll
        for (int q = 0; q < 3; ++q) *reinterpret_cast<u32x2*>(&b[q][row][2 * j]) = p[q];
    }
    // lane l: ranks 32 s + 8 (l / 16) + .. of row 16 q + l % 16
    __device__ __forceinline__ bf16x8 get(int part, int q, int s) const {
        const int lane = threadIdx.x & 63;
        return *reinterpret_cast<const bf16x8*>(&b[part][16 * q + (lane & 15)][64 * s + 16 * (lane >> 4)]);
    }
};

// First of a lane's eight columns in a wave's 128 from n0 on.
template <bool VEC>
__device__ __forceinline__ int lane_column(int n0) {
    return n0 + (VEC ? 8 : 1) * (threadIdx.x & 15);
}

// Weights of a wave's 128 columns, ranks 32 s to 32 s + 31, on their way to
// operands: rows of 64 bytes (or all r ranks, if fewer) are loaded as they lie,
// whole lines, and turned round in LDS.  put(): row 8 c + f (16 f + c where not VEC) at
// place (f, c); 16 bytes more per row and 32 per f keep the writes of neighbouring
// rows and the reads of 16 c in distinct banks.  get(f): lane l has ranks 8 (l /
// 16) + .. of column c = l % 16.
template <bool VEC>
struct Weights {
    static constexpr int row_bytes = 80, f_bytes = 16 * row_bytes + 32;
    u32x4 v[8];
    // A wave's share of LDS.
    struct Share {
        uint8_t b[8 * f_bytes];
    };
    // Chunks of 16 bytes of a row in step s, and at / chunks for at < 512.  FULL: four.
    template <bool FULL>
    static __device__ __forceinline__ int chunks_of(const LoraArgs& a, int s) { return FULL ? 4 : min(a.r - 32 * s, 32) / 8; }
    static __device__ __forceinline__ int row_of(int at, int chunks) {
        return at * (chunks == 4 ? 16384 : chunks == 3 ? 21846 : chunks == 2 ? 32768 : 65536) >> 16;
    }
    template <bool FULL>
    __device__ __forceinline__ void load_rows(const LoraArgs& a, int g, int n0, int s) {
        const int lane = a.tid & 63, chunks = chunks_of<FULL>(a, s);
        const uint16_t* from = a.b + static_cast<size_t>(g) * a.N * a.r + 32 * s;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (64 * i >= 128 * chunks) break;
            const int at = 64 * i + lane, row = row_of(at, chunks);
            v[i] = *reinterpret_cast<const u32x4*>(from + static_cast<size_t>(min(n0 + row, a.N - 1)) * a.r + 8 * (at - row * chunks));
        }
    }
    template <bool FULL>
    __device__ __forceinline__ void put_rows(const LoraArgs& a, int s, Share& to) const {
        const int lane = a.tid & 63, chunks = chunks_of<FULL>(a, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (64 * i >= 128 * chunks) break;
            const int at = 64 * i + lane, row = row_of(at, chunks);
            const int f = VEC ? row % 8 : row / 16, c = VEC ? row / 8 : row % 16;
            *reinterpret_cast<u32x4*>(to.b + f * f_bytes + c * row_bytes + 16 * (at - row * chunks)) = v[i];
        }
    }
    // Whether step s takes the way of four chunks, which does without branches (2048 tokens
    // x 4096 x 4096, us: rank 64 21.7 -> 21.2, rank 256 69 -> 58).  Not where both ways in
    // the code cost more: 64 tokens of 64 adapters at rank 16 8.2 -> 8.7, and, for want of
    // registers, 2048 tokens at rank 128 in fp32 42 -> 47 (in bf16 30.9 -> 30.3).  A kernel
    // of KS > 1 steps has more than 16 KS ranks.
    template <int KS>
    static __device__ __forceinline__ bool full(const LoraArgs& a, int s) {
        return KS != 1 && KS != 4 && (2 * (s + 1) <= KS || 32 * (s + 1) <= a.r);
    }
    template <int KS>
    __device__ __forceinline__ void load(const LoraArgs& a, int g, int n0, int s) {
        if (full<KS>(a, s)) load_rows<true>(a, g, n0, s);
        else load_rows<false>(a, g, n0, s);
    }
    template <int KS>
    __device__ __forceinline__ void put(const LoraArgs& a, int s, Share& to) const {
        if (full<KS>(a, s)) put_rows<true>(a, s, to);
        else put_rows<false>(a, s, to);
    }
    static __device__ __forceinline__ bf16x8 get(const LoraArgs& a, int s, const Share& from, int f) {
        const int lane = a.tid & 63, j = lane >> 4;
        // past r: any ranks, their v are zeros
        const int chunk = 32 * s + 8 * j < a.r ? j : 0;
        return *reinterpret_cast<const bf16x8*>(from.b + f * f_bytes + (lane & 15) * row_bytes + 16 * chunk);
    }
};

// The lane's four tokens of a tile of 16: rows of base and out, or -1.
struct Tokens {
    int t[4];
    __device__ __forceinline__ void load(const LoraArgs& a, const Run& run, int first) {
        const int at = first + 4 * (a.tid >> 4 & 3);
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = a.perm[min(at + i, a.T - 1)];
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = at + i < run.r1 && t[i] >= 0 && t[i] < a.T ? t[i] : -1;
    }
};

template <bool F32, bool VEC>
__device__ __forceinline__ void load_base(const LoraArgs& a, const Tokens& t, int n, Eight<F32, VEC> (&base)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) base[i].load(a.base, max(t.t[i], 0) * a.base_stride, n, a.N);
}

template <bool F32, bool VEC>
__device__ __forceinline__ void store_sum(const LoraArgs& a, const Tokens& t, int n, float scale, const f32x4 (&acc)[8],
                                          const Eight<F32, VEC> (&base)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (t.t[i] < 0) continue;
        float v[8];
#pragma unroll
        for (int f = 0; f < 8; ++f) v[f] = fmaf(scale, acc[f][i], base[i].value(f));
        store8<F32, VEC>(a.out, t.t[i] * a.out_stride, n, a.N, v);
    }
}

template <int ROWS, int KS>
__device__ __forceinline__ void add_products(const Parts<ROWS, KS>& v, const bf16x8 (&w)[8], int q, int s, f32x4 (&acc)[8]) {
#pragma unroll
    for (int p = 2; p >= 0; --p) {
        const bf16x8 t = v.get(p, q, s);
#pragma unroll
        for (int f = 0; f < 8; ++f) acc[f] = mfma16x16x32(t, w[f], acc[f]);
    }
}

// Rows of no adapter: base as it is, 128 columns of a wave.
template <bool F32, bool VEC>
__device__ __forceinline__ void copy_rows(const LoraArgs& a, const Run& run, int n0) {
    const int n = lane_column<VEC>(n0);
    for (int r = run.r0; r < run.r1; r += 16) {
        Tokens t;
        Eight<F32, VEC> base[4];
        t.load(a, run, r);
        load_base<F32, VEC>(a, t, n, base);
        hold_loads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (t.t[i] < 0) continue;
            float v[8];
#pragma unroll
            for (int f = 0; f < 8; ++f) v[f] = base[i].value(f);
            store8<F32, VEC>(a.out, t.t[i] * a.out_stride, n, a.N, v);
        }
    }
}

// The LDS of a workgroup of columns.
template <bool VEC, int KS>
struct Columns {
    Parts<kHalfRows, KS> parts;
    typename Weights<VEC>::Share shares[kWaves];
    int given_up;
};

// A wave's 128 columns from n0 on of the run's tokens.  TT: tiles of 16 tokens,
// KS: steps of 32 ranks.  flags: those of the n workgroups that make the tokens' v;
// with WAIT false v is there.  Not 0 if it gave up waiting, with nothing stored.
template <bool F32, bool VEC, int TT, int KS, bool WAIT>
__device__ __forceinline__ int make_columns(const LoraArgs& a, const Run& run, int n0, Columns<VEC, KS>& x,
                                             const unsigned long long* flags, int n) {
    auto& parts = x.parts;
    auto& share = x.shares[__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)];
    constexpr int kHeld = KS == 1 ? 1 : 2;     // steps' weights on their way
    constexpr int kTogether = KS == 1 ? 1 : TT;                // tiles whose sums are held over the steps
    const int col = lane_column<VEC>(n0);
    Weights<VEC> w[kHeld];
    Tokens t[TT];
    Eight<F32, VEC> base[TT][4];
#pragma unroll
    for (int s = 0; s < kHeld; ++s)
        if (32 * s < a.r) w[s].template load<KS>(a, run.g, n0, s);
#pragma unroll
    for (int q = 0; q < TT; ++q) t[q].load(a, run, run.r0 + 16 * q);
    const float scale = a.scales ? a.scales[run.g] : 1.f;
#pragma unroll
    for (int q = 0; q < TT; ++q) load_base<F32, VEC>(a, t[q], col, base[q]);
    w[0].template put<KS>(a, 0, share);
    if (KS > kHeld && 32 * kHeld < a.r) w[0].template load<KS>(a, run.g, n0, kHeld);
    hold_loads();
    if constexpr (WAIT) {
        if (threadIdx.x < kWave) {
            const bool there = wait_flags(flags, n, chain_tag(), a.polls);
            if (threadIdx.x == 0) x.given_up = !there;
        }
        __syncthreads();
        const int up = __builtin_amdgcn_readfirstlane(x.given_up);
        if (__builtin_expect(up != 0, 0)) return up;
    }
    // v, its parts of K added in order; zeros past the run and past r.  A thread has kMine
    // times four ranks, of which it asks for up to eight parts at once.
    constexpr int kQuads = 16 * TT * 8 * KS, kMine = (kQuads + kWaves * kWave - 1) / (kWaves * kWave);
    constexpr int kAtOnce = kMine < kMostSplits ? kMostSplits / kMine : 1;
    auto quad = [&](int i) { return i * kWaves * kWave + a.tid; };
    auto live = [&](int i) { return run.r0 + quad(i) / (8 * KS) < run.r1 && quad(i) % (8 * KS) * 4 < a.r; };
    f32x4 sum[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) sum[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s0 = 0; s0 < a.splits; s0 += kAtOnce) {
        u32x4 part[kAtOnce][kMine];
#pragma unroll
        for (int s = 0; s < kAtOnce; ++s) {
            if (s0 + s >= a.splits) break;
            const auto v = v_rows(a, run, s0 + s);
#pragma unroll
            for (int i = 0; i < kMine; ++i)
                part[s][i] = __builtin_amdgcn_raw_buffer_load_b128(
                    v, live(i) ? (quad(i) / (8 * KS) * a.r + quad(i) % (8 * KS) * 4) * 4 : 0, 0, kAuxDevice);
        }
#pragma unroll
        for (int s = 0; s < kAtOnce; ++s) {
            if (s0 + s >= a.splits) break;
#pragma unroll
            for (int i = 0; i < kMine; ++i) sum[i] += __builtin_bit_cast(f32x4, part[s][i]);
        }
    }
#pragma unroll
    for (int i = 0; i < kMine; ++i)
        if (kQuads % (kWaves * kWave) == 0 || quad(i) < kQuads)
            parts.set(quad(i) / (8 * KS), quad(i) % (8 * KS) * 4, live(i) ? sum[i] : f32x4{0.f, 0.f, 0.f, 0.f});
    __syncthreads();
#pragma unroll
    for (int q0 = 0; q0 < TT; q0 += kTogether) {
        f32x4 acc[kTogether][8];
#pragma unroll
        for (int q = 0; q < kTogether; ++q)
#pragma unroll
            for (int f = 0; f < 8; ++f) acc[q][f] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            if (32 * s >= a.r) break;
            // the wave's own share: no barrier
            if (s) {
                wave_lds_fence();
                w[s % kHeld].template put<KS>(a, s, share);
                wave_lds_fence();
                if (KS > kHeld && 32 * (s + kHeld) < a.r) w[s % kHeld].template load<KS>(a, run.g, n0, s + kHeld);
                if (KS > kHeld) hold_loads();
            }
            bf16x8 wo[8];
#pragma unroll
            for (int f = 0; f < 8; ++f) wo[f] = Weights<VEC>::get(a, s, share, f);
#pragma unroll
            for (int q = 0; q < kTogether; ++q) add_products(parts, wo, q0 + q, s, acc[q]);
        }
#pragma unroll
        for (int q = 0; q < kTogether; ++q) store_sum<F32, VEC>(a, t[q0 + q], col, scale, acc[q], base[q0 + q]);
    }
    asm volatile("");                          // the stores' branches end here, not in the return
    return 0;
}

// Tile `at` of columns after make_columns gave up: v by this workgroup, 16 ranks of
// 16 tokens at a time, then the columns.  The same bits, whatever the tile, v's at the
// place where their maker stores them too.
template <bool F32, bool VEC, int KS>
__device__ __forceinline__ void columns_alone(LoraArgs& a, int at, int n_tiles, Columns<VEC, KS>& x) {
    // nothing that follows from these is held from before: there would be too few registers
    asm volatile("" : "+v"(a.tid), "+s"(at), "+s"(n_tiles));
    Run run = load_half(a, at / n_tiles);
    const int n0 = at % n_tiles * kCols + 128 * __builtin_amdgcn_readfirstlane(a.tid >> 6), end = run.r1;
    for (; run.r0 < end; run.r0 += 16) {
        run.r1 = min(end, run.r0 + 16);
        __syncthreads();                       // LDS is free
        for (int i = 0, blocks = ceil_div(a.r, 16); i < a.splits * blocks; ++i) {
            asm volatile("" : "+v"(a.tid));
            make_v<1, 1>(a, run, i / blocks, i % blocks * 16, reinterpret_cast<f32x4*>(&x));
            __syncthreads();
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");       // v is there when all threads are past the barrier
        __syncthreads();
        asm volatile("" : "+v"(a.tid));
        make_columns<F32, VEC, 1, KS, false>(a, run, n0, x, nullptr, 0);
    }
}

// Workgroups go round the XCDs, whose L2s are apart.  With several blocks of ranks
// those of two neighbouring halves are on one XCD, so that it alone reads their x, and their
// a mostly once (2048 tokens of 8 requests x 4096 x 4096, us: rank 64 22.3 -> 21.1, rank
// 128 34.4 -> 31.0, rank 256 58.9 -> 58.1; 512 of 64 adapters, rank 64, 2048 columns, 16.8 ->
// 16.1; with four neighbours rank 64 as slow as without): `big` workgroups are those of 8
// kNear halves.  The count is that of all halves the schedule has room for; where few of
// them have tokens, their makers share few XCDs, and from rank 128 on that costs more than
// the order gains (64 tokens of 8 requests, rank 128, 14.5 -> 17.7, in fp32 16.3 -> 19.6;
// 32 of one, 12.5 -> 14.9; 8 of one, rank 64, 7.6 -> 7.5, rank 256 12.4 -> 18.6).
constexpr int kXcds = 8, kNear = 2;
__host__ __device__ inline bool near_halves(int halves, int ranks) { return ranks > 1 && halves >= kXcds * kNear; }
__host__ __device__ inline long long lora_makers(long long halves, int each, bool near) {
    return near ? (halves + kXcds * kNear - 1) / (kXcds * kNear) * (kXcds * kNear) * each : halves * each;
}

// The grid: `ranks` blocks of 32 ranks x a.splits parts of K of every half item,
// then n_tiles tiles of columns of every half item.  Halves without tokens end at once,
// but are dispatched, and the parts of K are fewer for them (2048 tokens of 8 requests, us:
// rank 32, of 16 adapters 16.8, of 64 18.5, of 1024 23.3; rank 128 30.2, 30.6, 47.7).
//
// LDS: 48.5 / 54.5 / 66.5 / 90.5 KB for KS = 1 / 2 / 4 / 8, most of it v in three parts,
// so that a CU of 160 KB has 3 / 2 / 2 / 1 workgroups; those that make v have the
// same though they use 16 KB.  That is what bounds high ranks: at KS = 8 a SIMD has one wave.
//
// A workgroup of columns follows those that make its v in the grid, so alone on the
// GPU it waits for what runs already.  Beside another such launch it may wait for
// what does not: of each, columns can hold all of an XCD on which the other's makers
// have no place yet.  So a wait ends after a.polls polls, the workgroup makes v itself,
// and no launch depends on another's progress.
template <bool F32, bool VEC, int KS>
__global__ __launch_bounds__(kWaves* kWave, KS == 1 ? 3 : KS <= 4 ? 2 : 1) void lora_kernel(LoraArgs args, int n_tiles, int ranks) {
    LoraArgs a = args;
    a.tid = threadIdx.x;
    constexpr size_t kPartBytes = kWaves * 4 * kWave * sizeof(f32x4);
    __shared__ __align__(16) uint8_t lds[sizeof(Columns<VEC, KS>) > kPartBytes ? sizeof(Columns<VEC, KS>) : kPartBytes];
    const int each = a.splits * ranks, halves = a.n_items * kHalves;
    const bool near = near_halves(halves, ranks);
    const int makers = lora_makers(halves, each, near);
    int at = blockIdx.x;
    if (at < makers) {
        if (near) {
            const int big = kXcds * kNear * each, in = at % big, k = in / kXcds;
            const int half = (at / big * kXcds + in % kXcds) * kNear + k / each;
            if (half >= halves) return;
            at = half * each + k % each;
        }
        const Run run = load_half(a, at / each);
        if (run.g < 0 || run.g == a.L) return;
        f32x4* part = reinterpret_cast<f32x4*>(lds);
        const int split = at % each / ranks, j0 = at % ranks * 32, rows = run.r1 - run.r0;
        if (a.r <= 16) {
            if (rows > 16) make_v<1, 2>(a, run, split, j0, part);
            else make_v<1, 1>(a, run, split, j0, part);
        } else {
            if (rows > 16) make_v<2, 2>(a, run, split, j0, part);
            else make_v<2, 1>(a, run, split, j0, part);
        }
        raise_flag(a.flags + at, chain_tag());
        return;
    }
    at -= makers;
    const int half = at / n_tiles;
    const Run run = load_half(a, half);
    if (run.g < 0) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = at % n_tiles * kCols + 128 * wave;
    if (run.g == a.L) {
        if (!a.in_place && n0 < a.N) copy_rows<F32, VEC>(a, run, n0);
        return;
    }
    Columns<VEC, KS>& x = *reinterpret_cast<Columns<VEC, KS>*>(lds);
    const unsigned long long* flags = a.flags + static_cast<size_t>(half) * each;
    int given_up = run.r1 - run.r0 > 16 ? make_columns<F32, VEC, 2, KS, true>(a, run, n0, x, flags, each)
                                        : make_columns<F32, VEC, 1, KS, true>(a, run, n0, x, flags, each);
    // The ways meet here in one value that the compiler knows nothing of, and the rare one
    // lies behind the others' code.  With a return of their own instead, the registers of
    // both were held over each other and spilled (5 tokens at rank 16 6.6 -> 7.5 us); so
    // 64 tokens of 64 at rank 16 take 8.0 us with and without this way, 5 tokens 6.75 and 6.6.
    given_up = __builtin_amdgcn_readfirstlane(given_up);
    asm volatile("" : "+s"(given_up));
    if (__builtin_expect(given_up != 0, 0)) columns_alone<F32, VEC, KS>(a, at, n_tiles, x);
}

// Up to four tokens, every workgroup with the whole of their v (4096 x 4096 at
// rank 16, us: one token 4.7, of which a launch that does nothing is 2.2, with v handed
// over 6.4).  No matrix instruction, whose operands would be turned round for the sake of
// 16 rows: loads as Sums', of which a lane takes the dot products with its 8 values of
// each token, two values an instruction (off by at most 2^-22.5 of the magnitudes,
// measured).  The lanes of a quad are added by lane exchanges, what else a row has in
// LDS, in order.  Then a thread has two columns.
template <bool F32, int RF, int NT>
__device__ __forceinline__ void few_body(const LoraArgs& a, const Run& run, int n0, float* part, float* sums) {
    constexpr int kRanks = 16 * RF, kAhead = RF == 1 ? 4 : 2, kEach = kFewCols / (kFewWaves * kWave);
    using S = Sums<RF, 1, 1>;
    const int lane = threadIdx.x & 63, row = lane & 12;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), steps = ceil_div(a.K, kStep);
    const int beg = steps * wave / kFewWaves, end = steps * (wave + 1) / kFewWaves;
    const uint16_t* arow = a.a + static_cast<size_t>(run.g) * a.r * a.K;
    int aoff[RF], t[NT];
#pragma unroll
    for (int f = 0; f < RF; ++f) aoff[f] = min(16 * f + row, a.r - 4) * a.K;
#pragma unroll
    for (int q = 0; q < NT; ++q) t[q] = __builtin_amdgcn_readfirstlane(a.perm[min(run.r0 + q, run.r1 - 1)]);
    u32x4 av[kAhead][RF][4], xv[kAhead][NT];
    const uint16_t* xrow[NT];
    auto load_a = [&](int s) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int f = 0; f < RF; ++f)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    av[u][f][i] = *reinterpret_cast<const u32x4*>(arow + i * a.K + (aoff[f] + S::place(a, s + u, end)));
    };
    auto load_x = [&](int s) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int q = 0; q < NT; ++q) xv[u][q] = *reinterpret_cast<const u32x4*>(xrow[q] + S::place(a, s + u, end));
    };
    load_a(beg);
#pragma unroll
    for (int q = 0; q < NT; ++q) {
        const bool sound = run.r0 + q < run.r1 && t[q] >= 0 && t[q] < a.T;
        t[q] = sound ? t[q] : -1;
        xrow[q] = a.x + max(t[q], 0) * a.x_stride;
    }
    load_x(beg);
    // the thread's columns: weights and base
    u32x4 w[kEach][2 * RF];
    uint32_t base[kEach][NT];
#pragma unroll
    for (int c = 0; c < kEach; ++c) {
        const int n = min(n0 + c * kFewWaves * kWave + static_cast<int>(threadIdx.x), a.N - 1);
        const uint16_t* b = a.b + (static_cast<size_t>(run.g) * a.N + n) * a.r;
#pragma unroll
        for (int h = 0; h < 2 * RF; ++h) w[c][h] = *reinterpret_cast<const u32x4*>(b + (8 * h < a.r ? 8 * h : 0));
#pragma unroll
        for (int q = 0; q < NT; ++q) {
            const long long at = max(t[q], 0) * a.base_stride + n;
            base[c][q] = F32 ? static_cast<const uint32_t*>(a.base)[at] : static_cast<const uint16_t*>(a.base)[at] << 16;
        }
    }
    const float scale = a.scales ? a.scales[run.g] : 1.f;
    hold_loads();

    f32x4 acc[RF][NT];
#pragma unroll
    for (int f = 0; f < RF; ++f)
#pragma unroll
        for (int q = 0; q < NT; ++q) acc[f][q] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s = beg; s < end; s += kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (s + u >= end) break;
            if (kStep * (s + u + 1) > a.K && kStep * (s + u) + S::lane_k() >= a.K) {
#pragma unroll
                for (int q = 0; q < NT; ++q) xv[u][q] = u32x4{0u, 0u, 0u, 0u};
            }
#pragma unroll
            for (int f = 0; f < RF; ++f)
#pragma unroll
                for (int q = 0; q < NT; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int d = 0; d < 4; ++d) {
                            const uint32_t w2 = av[u][f][i][d], x2 = xv[u][q][d];
                            acc[f][q][i] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w2), __builtin_bit_cast(bf16x2, x2),
                                                                           acc[f][q][i], false);
                        }
        }
        if (s + kAhead < end) {
            load_a(s + kAhead);
            load_x(s + kAhead);
            hold_loads();
        }
    }
    // [wave and piece][token][rank]
#pragma unroll
    for (int f = 0; f < RF; ++f)
#pragma unroll
        for (int q = 0; q < NT; ++q) {
            f32x4 v = acc[f][q];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v[i]), 0xB1, 0xf, 0xf, true));
                v[i] += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v[i]), 0x4E, 0xf, 0xf, true));
            }
            if (!(lane & 3)) *reinterpret_cast<f32x4*>(part + ((4 * wave + (lane >> 4)) * NT + q) * kRanks + 16 * f + row) = v;
        }
    __syncthreads();
    if (threadIdx.x < NT * kRanks) {
        float v = 0.f;
#pragma unroll
        for (int p = 0; p < 4 * kFewWaves; ++p) v += part[p * NT * kRanks + threadIdx.x];
        sums[threadIdx.x] = static_cast<int>(threadIdx.x) % kRanks < a.r ? v : 0.f;
    }
    __syncthreads();
    float o[kEach][NT];
#pragma unroll
    for (int c = 0; c < kEach; ++c)
#pragma unroll
        for (int q = 0; q < NT; ++q) o[c][q] = 0.f;
#pragma unroll
    for (int h = 0; h < 2 * RF; ++h) {
        if (8 * h >= a.r) break;
#pragma unroll
        for (int q = 0; q < NT; ++q) {
            const f32x4 lo = *reinterpret_cast<const f32x4*>(sums + q * kRanks + 8 * h);
            const f32x4 hi = *reinterpret_cast<const f32x4*>(sums + q * kRanks + 8 * h + 4);
#pragma unroll
            for (int c = 0; c < kEach; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t b = w[c][h][i];
                    o[c][q] = fmaf(bf16lo(b), i < 2 ? lo[2 * i] : hi[2 * i - 4], o[c][q]);
                    o[c][q] = fmaf(bf16hi(b), i < 2 ? lo[2 * i + 1] : hi[2 * i - 3], o[c][q]);
                }
        }
    }
#pragma unroll
    for (int c = 0; c < kEach; ++c) {
        const int n = n0 + c * kFewWaves * kWave + threadIdx.x;
#pragma unroll
        for (int q = 0; q < NT; ++q) {
            if (t[q] < 0 || n >= a.N) continue;
            const float v = fmaf(scale, o[c][q], __uint_as_float(base[c][q]));
            const long long at = t[q] * a.out_stride + n;
            if constexpr (F32) static_cast<float*>(a.out)[at] = v;
            else static_cast<uint16_t*>(a.out)[at] = static_cast<uint16_t>(bf16_pair(v, v));
        }
    }
}

template <bool F32, int RF>
__global__ __launch_bounds__(kFewWaves* kWave) void lora_few_kernel(LoraArgs args, int n_tiles) {
    LoraArgs a = args;
    a.tid = threadIdx.x;
    __shared__ __align__(16) float part[4 * kFewWaves * 4 * 16 * RF];
    __shared__ __align__(16) float sums[4 * 16 * RF];
    Run run = load_run(a, blockIdx.x / n_tiles);
    if (run.g < 0) return;
    const int n0 = blockIdx.x % n_tiles * kFewCols;
    if (run.g == a.L) {
        if (!a.in_place) {
            const int wave = threadIdx.x >> 6;
            copy_rows<F32, false>(a, run, n0 + 128 * wave);
        }
        return;
    }
    const int rows = run.r1 - run.r0;          // at most a.T
    if (rows == 1) few_body<F32, RF, 1>(a, run, n0, part, sums);
    else if (rows == 2) few_body<F32, RF, 2>(a, run, n0, part, sums);
    else few_body<F32, RF, 4>(a, run, n0, part, sums);
}

template <bool F32>
hipError_t launch_few(const LoraArgs& a, hipStream_t st) {
    const int n_tiles = ceil_div(a.N, kFewCols), blocks = a.n_items * n_tiles;
    if (a.r <= 16) lora_few_kernel<F32, 1><<<blocks, kFewWaves * kWave, 0, st>>>(a, n_tiles);
    else lora_few_kernel<F32, 2><<<blocks, kFewWaves * kWave, 0, st>>>(a, n_tiles);
    return hipGetLastError();
}

template <bool F32, bool VEC>
hipError_t launch(const LoraArgs& a, hipStream_t st) {
    const int n_tiles = ceil_div(a.N, kCols), ranks = ceil_div(a.r, 32), halves = a.n_items * kHalves;
    const int blocks = lora_makers(halves, a.splits * ranks, near_halves(halves, ranks)) + halves * n_tiles;
    if (a.r <= 32) lora_kernel<F32, VEC, 1><<<blocks, kWaves * kWave, 0, st>>>(a, n_tiles, ranks);
    else if (a.r <= 64) lora_kernel<F32, VEC, 2><<<blocks, kWaves * kWave, 0, st>>>(a, n_tiles, ranks);
    else if (a.r <= 128) lora_kernel<F32, VEC, 4><<<blocks, kWaves * kWave, 0, st>>>(a, n_tiles, ranks);
    else lora_kernel<F32, VEC, 8><<<blocks, kWaves * kWave, 0, st>>>(a, n_tiles, ranks);
    return hipGetLastError();
}

}  // namespace

// Few tokens: see few_body (us, and with v handed over, 4096 x 4096: rank 16, one token
// 4.7, 6.4; four 4.9, 6.8, of one adapter 6.7, 7.0; rank 32, one 6.2, 6.4; two 6.3, 6.9, of
// one adapter 6.8, 6.6; four 6.7, 7.0, of one adapter 9.1, 7.1; one at rank 64 11.3, 7.2).
// The time of v in each workgroup grows with K, which the rule leaves out: one token
// at K = 1024 4.4, 5.7, at 14336 8.1, 7.5, at 28672 11.5, 8.7; at rank 32 5.1, 5.8, 11.2, 8.1
// and 23, 10.
// Else parts of K until the workgroups that make v are about one and a half a CU (us, and
// with twice as many, 4096 x 4096: 512 tokens of 64 adapters, rank 64, 2048 columns, 16.1,
// 16.9; 2048 of 8 requests at rank 32 16.8, 16.4, at 64 21.1, 22.9, at 128 30.9, 33.2), with a
// step or more for each wave.  The guess of the runs is of adapters that are mostly in use:
// of 1024 of which 8 are, rank 32 gets one part of K in place of four.
LoraShape lora_shape(int T, int K, int N, int r, int L) {
    LoraShape p{0, 0, 0};
    if (r <= 32 && T * ceil_div(r, 16) <= 4) return p;
    const int groups = L < T ? L : T, steps = ceil_div(K, kStep), ranks = ceil_div(r, 32);
    const int runs = ceil_div(T, kHalfRows) + groups / 2;      // taking it that half of the adapters end in a partial run
    p.splits = 1;
    while (p.splits < kMostSplits && 2ll * p.splits * runs * ranks <= 380 && steps >= 2 * p.splits * kWaves) p.splits *= 2;
    const long long halves = static_cast<long long>(plan_items(T, L)) * kHalves;
    p.flags = halves * p.splits * ranks;
    p.blocks = lora_makers(halves, p.splits * ranks, near_halves(halves, ranks)) + halves * ((static_cast<long long>(N) + kCols - 1) / kCols);
    return p;
}

hipError_t launch_lora_add(const LoraArgs& a, hipStream_t st) {
    if (!a.splits) return a.f32 ? launch_few<true>(a, st) : launch_few<false>(a, st);
    if (a.f32) return a.vec ? launch<true, true>(a, st) : launch<true, false>(a, st);
    return a.vec ? launch<false, true>(a, st) : launch<false, false>(a, st);
}

}  // namespace qrmoe
