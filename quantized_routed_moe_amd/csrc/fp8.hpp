// Shared parts of the FP8 operators (include/moe_fp8.h): kernel arguments,
// the row schedule of a grouped product, E4M3 conversions and the launch
// interface between the entry points (fp8.hip) and the kernels.
#pragma once

#include "chain.hpp"
#include "common.hpp"

namespace qrmoe {

constexpr int kRun = 128;                    // values that share a scale
constexpr float kE4m3Max = 448.f;
constexpr float kScaleMin = 1.17549435e-38f;  // 2^-126, the smallest scale

struct Fp8Args {
    int R, E, N, K;               // rows, experts (1: dense), weight rows of a matrix, depth
    const uint8_t* a;             // E4M3 [a_rows][K], rows a_stride bytes apart
    long long a_stride;
    int a_rows;
    const float* a_scales;        // [a_rows][ceil(K/128)]
    const uint8_t* w[2];          // [E][N][K]; gate/up: both, else w[0]
    const float* w_scales[2];     // [E][ceil(N/128)][ceil(K/128)]
    const int32_t* offsets;       // [E+1], or null: one group of R rows
    const int32_t* perm;          // [R], or null: row r reads a[r]
    int k;
    void* out;                    // [R][N], rows out_stride values apart
    long long out_stride;
    int out_f32;                  // 1: fp32, 0: bf16
    int out_vec;                  // 1: four consecutive values can be stored at once
    uint8_t* act;                 // gate/up: E4M3 [R][N] ...
    float* act_scales;            // ... and its scales [R][ceil(N/128)]
    float* hidden;                // gate/up by workgroups of less than 128 columns: silu(g) * u in fp32
                                  // [R][N] (workspace) ...
    unsigned long long* flags;    // ... and a flag per workgroup
};

// Rows [r0, r1) of expert e; e = E: rows of no expert, to be zeroed; e = -1
// past the last item.
struct RowItem {
    int e, r0, r1;
};

// Item idx of the schedule that cuts every expert's rows into runs of at
// most `rows`, experts in id order, and after them (rest) the rows of no expert,
// below offsets[0] and from offsets[E] on, whose zeros so are spread over the
// grid as the products are (16384 rows x 4096 in fp32, 64 of them live: 41 us; by
// the workgroups of the first item 1280).  Lane e of the calling wave reads
// expert e's bounds (clamped to [0, R], so no offset is followed out of range)
// and a wave scan over the experts' item counts finds the owner.  Uniform.
__device__ __forceinline__ RowItem row_item(const Fp8Args& a, int idx, int rows, bool rest) {
    if (!a.offsets) {
        const int r0 = idx * rows;
        return RowItem{r0 < a.R ? 0 : -1, r0, min(a.R, r0 + rows)};
    }
    const int lane = threadIdx.x & 63;
    int lo = 0, hi = 0;
    if (lane < a.E) {
        lo = min(max(a.offsets[lane], 0), a.R);
        hi = min(max(a.offsets[lane + 1], lo), a.R);
    }
    const int items = (hi - lo + rows - 1) / rows;
    int incl = items;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(incl, o);
        if (lane >= o) incl += v;
    }
    const uint64_t hit = __ballot(idx >= incl - items && idx < incl);
    if (!hit) {
        if (!rest) return RowItem{-1, 0, 0};
        const int head = min(max(a.offsets[0], 0), a.R), tail = min(max(a.offsets[a.E], head), a.R);
        const int head_items = (head + rows - 1) / rows, at = idx - lane_value(incl, 63);
        const long long r0 = at < head_items ? static_cast<long long>(at) * rows
                                             : tail + static_cast<long long>(at - head_items) * rows;
        const int r1 = at < head_items ? head : a.R;
        if (r0 >= r1) return RowItem{-1, 0, 0};
        return RowItem{a.E, static_cast<int>(r0), static_cast<int>(min(r0 + rows, static_cast<long long>(r1)))};
    }
    const int e = __ffsll(static_cast<unsigned long long>(hit)) - 1;
    const int r0 = lane_value(lo, e) + (idx - lane_value(incl - items, e)) * rows;
    return RowItem{e, r0, min(lane_value(hi, e), r0 + rows)};
}

// Upper bound of the items of any sound offsets.
inline long long row_items(const Fp8Args& a, int rows, bool rest) {
    if (!a.offsets) return (static_cast<long long>(a.R) + rows - 1) / rows;
    const long long groups = a.E + (rest ? 2 : 0);
    return (a.R + (groups < a.R ? groups : a.R) * (rows - 1)) / rows;      // each group's last run as short as can be
}

// Row of `a` that sorted row r reads.
__device__ __forceinline__ int source_row(const Fp8Args& a, int r) {
    const int s = a.perm ? a.perm[r] / a.k : r;
    return min(max(s, 0), a.a_rows - 1);
}

// Zeros in the rows of an item and COLS columns from n0 on.
template <int COLS>
__device__ __forceinline__ void zero_tile(const Fp8Args& a, const RowItem& it, int n0) {
    constexpr int kChunks = COLS / 4;
    for (int i = threadIdx.x; i < (it.r1 - it.r0) * kChunks; i += blockDim.x) {
        const int n = n0 + 4 * (i % kChunks);
        const long long at = (it.r0 + i / kChunks) * a.out_stride + n;
        if (a.out_vec && n + 4 <= a.N) {
            if (a.out_f32) *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + at) = f32x4{0.f, 0.f, 0.f, 0.f};
            else *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + at) = u32x2{0u, 0u};
        } else {
            for (int c = 0; c < 4 && n + c < a.N; ++c) {
                if (a.out_f32) static_cast<float*>(a.out)[at + c] = 0.f;
                else static_cast<uint16_t*>(a.out)[at + c] = 0;
            }
        }
    }
}

// Floats that no kernel writes while this one runs, read through the scalar
// cache: a wave's block scales are one value for all lanes.
typedef const __attribute__((address_space(4))) float Scalar;
__device__ __forceinline__ Scalar* scalar_ptr(const float* p) {
    return reinterpret_cast<Scalar*>(reinterpret_cast<uintptr_t>(p));
}

// Memory from p on, for copies by a 32-bit lane offset and a scalar offset
// (raw 32-bit data, no stride; every offset is inside the tensor).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const uint8_t* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, 0xffffffffu, 4 << 15);
}

__device__ __forceinline__ void store_hidden(const Fp8Args& a, int r, int n, float v) {
    __hip_atomic_store(a.hidden + static_cast<size_t>(r) * a.N + n, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Eight E4M3 codes -> bf16, exact (E4M3 has 4 significant bits and an
// exponent range inside bf16's).
__device__ __forceinline__ bf16x8 e4m3x8_to_bf16(uint32_t lo, uint32_t hi) {
    const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false);
    const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true);
    const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false);
    const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true);
    return bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// Four values, already divided by their scale, to E4M3 codes (low byte
// first).  The scale makes every finite magnitude at most 448 (1 + 2^-22),
// which rounds to 448, so there is no clamp and a NaN stays a NaN.
__device__ __forceinline__ uint32_t e4m3x4_rne(float a, float b, float c, float d) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
}

__device__ __forceinline__ float run_scale(float amax) { return fmaxf(amax / kE4m3Max, kScaleMin); }

// Gate/up by workgroups of COLS < 128 columns: every workgroup has stored its
// silu(g) u (store_hidden); the one that finishes a run of 128 columns turns
// it into E4M3.  Each raises its own flag (a value unique to the launch, see
// chain.hpp, so nothing has to be cleared) once its stores are acknowledged,
// and reads the flags of the run's workgroups once that store is acknowledged
// too: whichever flag is acknowledged last, its workgroup sees them all.  When
// several do, they store the same bytes.  Nobody waits for another.
template <int COLS>
__device__ __forceinline__ void finish_run(const Fp8Args& a, const RowItem& it, int item, int n_tile, int n_tiles, int* lds) {
    constexpr int kPer = kRun / COLS;               // workgroups of a run
    const unsigned long long tag = chain_tag();
    unsigned long long* flags = a.flags + static_cast<size_t>(item) * n_tiles;
    raise_flag(flags + n_tile, tag);
    const int run = n_tile / kPer, lane = threadIdx.x & 63;
    if (threadIdx.x < kWave) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        const int other = run * kPer + lane;
        const bool there = lane >= kPer || other >= n_tiles ||
                           __hip_atomic_load(flags + other, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == tag;
        const bool all = __all(there);
        if (lane == 0) *lds = all;
    }
    __syncthreads();
    if (!*lds) return;
    const int NB = (a.N + kRun - 1) / kRun, n = run * kRun + 2 * lane;
    const bool live = n < a.N;                      // N is a multiple of 32
    for (int r = it.r0 + (threadIdx.x >> 6); r < it.r1; r += blockDim.x >> 6) {
        float v0 = 0.f, v1 = 0.f;
        if (live) {
            const unsigned long long v =
                __hip_atomic_load(reinterpret_cast<const unsigned long long*>(a.hidden + static_cast<size_t>(r) * a.N + n),
                                  __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            v0 = __uint_as_float(static_cast<uint32_t>(v));
            v1 = __uint_as_float(static_cast<uint32_t>(v >> 32));
        }
        float m = fmaxf(fabsf(v0), fabsf(v1));
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
        const float s = run_scale(m);
        if (live)
            *reinterpret_cast<uint16_t*>(a.act + static_cast<size_t>(r) * a.N + n) =
                static_cast<uint16_t>(e4m3x4_rne(v0 / s, v1 / s, 0.f, 0.f));
        if (lane == 0) a.act_scales[static_cast<size_t>(r) * NB + run] = s;
    }
}

// How a call is cut into workgroups.  `cols` output columns x `rows` token
// rows of one expert each.
enum class Fp8Path {
    kFew,    // 16 columns x 16 rows, the depth split over 8 waves (fp8_few.hip)
    kMid,    // 64 columns (gate/up 32) x 64 rows, 4 waves (fp8_tile.hip)
    kMany    // 256 columns (gate/up 128) x 128 rows, 8 waves (fp8_tile.hip)
};

struct Fp8Plan {
    Fp8Path path;
    int cols, rows, n_tiles;
    int group_bits;       // kMid, kMany: 2^group_bits groups of column tiles are dealt to the XCDs
    int items;            // upper bound, with those of no expert's rows; the grid may be rounded up beyond it
    int products;         // upper bound of those that have a product to do
    long long blocks;
};

// A grid holds fewer than 2^32 threads, and no workgroup here has more than 512.
constexpr long long kMostBlocks = 1ll << 23;

inline Fp8Plan fp8_plan(const Fp8Args& a, bool gate_up) {
    Fp8Plan p;
    // Workgroups of the small tiles, taking it that every expert that can have
    // rows has some and that half of the experts end in a partial run of rows.
    // Measured on both sides (us; T tokens, two of E experts of 4096 x 2048
    // each): kFew while a CU gets few of its workgroups (32 x 4096 x 4096: 11.9,
    // kMid 16.0; 64 rows 20.6, 20.1; gate/up, E = 8, T = 32: 29, 29; T = 64:
    // 50, 30), the rows of a dense product are four or fewer (x 65536 x 4096: one
    // row 48, 59, kMany 66; four 54, 59; eight 65, 59) or an expert has a row or
    // two (E = 64, T = 64: 171, 199, kMany 171).  Then kMid until its workgroups
    // make two and a half rounds of two per CU (1024 x 4096 x 4096: 56, kMany 64;
    // 512 rows: 29, 62; down, E = 8, T = 256: 32, 35; T = 1024: 65, 55), or one
    // with both gate and up (E = 8, T = 128: 39, 47; T = 256: 81, 68).
    const int cols = gate_up ? 128 : 256;
    const long long experts = a.offsets ? (a.E < a.R ? a.E : a.R) : 1;
    auto items = [&](int rows) {
        const long long runs = a.offsets ? a.R / rows + experts / 2 : (static_cast<long long>(a.R) + rows - 1) / rows;
        return runs > experts ? runs : experts;
    };
    const long long few = items(16) * ((a.N + 15) / 16), mid_cols = gate_up ? 32 : 64;
    const long long mid = items(64) * ((a.N + mid_cols - 1) / mid_cols);
    const long long few_blocks = row_items(a, 16, !gate_up) * ((a.N + 15) / 16);
    p.path = few <= 1024 || (a.R <= (a.offsets ? 2 * experts : 4) && few_blocks < kMostBlocks) ? Fp8Path::kFew
             : mid <= (gate_up ? 512 : 1280)                                                 ? Fp8Path::kMid
                                                                                             : Fp8Path::kMany;
    p.cols = p.path == Fp8Path::kFew ? 16 : p.path == Fp8Path::kMid ? (gate_up ? 32 : 64) : cols;
    p.rows = p.path == Fp8Path::kFew ? 16 : p.path == Fp8Path::kMid ? 64 : 128;
    p.n_tiles = (a.N + p.cols - 1) / p.cols;
    p.items = static_cast<int>(row_items(a, p.rows, !gate_up));
    p.products = static_cast<int>(row_items(a, p.rows, false));
    // Four groups of column tiles where they come out even, and as many as it
    // takes that no XCD is without a product (17 x 128256 x 4096, 501 tiles of one
    // item: 128 us, with one group, that is on one XCD, 500).
    p.group_bits = p.n_tiles % 4 == 0 ? 2 : p.n_tiles % 2 == 0 ? 1 : 0;
    while ((8 >> p.group_bits) > p.products) ++p.group_bits;
    const int groups = 1 << p.group_bits, classes = 8 / groups, per = (p.n_tiles + groups - 1) / groups;
    p.blocks = p.path == Fp8Path::kFew ? static_cast<long long>(p.n_tiles) * p.items
                                       : 8ll * per * ((p.items + classes - 1) / classes);
    return p;
}

// Workspace of a gate/up call: hidden, then the flags of the most workgroups
// that the paths with a hidden have.
inline size_t fp8_hidden_bytes(const Fp8Args& a) { return (static_cast<size_t>(a.R) * a.N * 4 + 255) / 256 * 256; }
inline size_t fp8_flag_bytes(const Fp8Args& a) {
    return (static_cast<size_t>((a.N + 15) / 16) * row_items(a, 16, false) * 8 + 255) / 256 * 256;
}

hipError_t launch_fp8_few(const Fp8Args& a, const Fp8Plan& p, bool gate_up, hipStream_t st);
hipError_t launch_fp8_tile(const Fp8Args& a, const Fp8Plan& p, bool gate_up, hipStream_t st);

struct NormArgs {
    int T, d;
    const void *x, *res, *weight;
    void* res_out;
    long long x_stride, res_stride, res_out_stride;
    float eps;
    uint16_t* y;
    uint8_t* q;
    float* q_scales;
};
hipError_t launch_add_rmsnorm(const NormArgs& a, bool x_f32, bool res_f32, bool w_f32, hipStream_t st);

}  // namespace qrmoe
