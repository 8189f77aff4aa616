// Shared parts of the FP8 operators (include/moe_fp8.h): kernel arguments,
// the row schedule of a grouped product, E4M3 conversions and the launch
// interface between the entry points (fp8.hip) and the kernels.
#pragma once

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
    float* hidden;                // gate/up of few rows: silu(g) * u in fp32 [R][N]
    uint8_t* act;                 // gate/up of many rows: E4M3 [R][N] ...
    float* act_scales;            // ... and its scales [R][ceil(N/128)]
};

// Rows [r0, r1) of expert e; e = -1 past the last item.
struct RowItem {
    int e, r0, r1;
};

// Item idx of the schedule that cuts every expert's rows into runs of at
// most `rows`, experts in id order.  Lane e of the calling wave reads expert
// e's bounds (clamped to [0, R], so no offset is followed out of range) and
// a wave scan over the experts' item counts finds the owner.  Uniform.
__device__ __forceinline__ RowItem row_item(const Fp8Args& a, int idx, int rows) {
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
    if (!hit) return RowItem{-1, 0, 0};
    const int e = __ffsll(static_cast<unsigned long long>(hit)) - 1;
    const int r0 = lane_value(lo, e) + (idx - lane_value(incl - items, e)) * rows;
    return RowItem{e, r0, min(lane_value(hi, e), r0 + rows)};
}

// Upper bound of the items of any offsets.
inline long long row_items(const Fp8Args& a, int rows) {
    if (!a.offsets) return (static_cast<long long>(a.R) + rows - 1) / rows;
    return a.R / rows + (a.E < a.R ? a.E : a.R);
}

// Row of `a` that sorted row r reads.
__device__ __forceinline__ int source_row(const Fp8Args& a, int r) {
    const int s = a.perm ? a.perm[r] / a.k : r;
    return min(max(s, 0), a.a_rows - 1);
}

// Rows at or past offsets[E], columns [n0, n1): zeros.
__device__ __forceinline__ void zero_rows_past_end(const Fp8Args& a, int n0, int n1) {
    const int first = min(max(a.offsets[a.E], 0), a.R);
    const int cols = n1 - n0;
    for (long long i = threadIdx.x; i < static_cast<long long>(a.R - first) * cols; i += blockDim.x) {
        const long long at = (first + i / cols) * a.out_stride + n0 + i % cols;
        if (a.out_f32) static_cast<float*>(a.out)[at] = 0.f;
        else static_cast<uint16_t*>(a.out)[at] = 0;
    }
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

// Output columns of one workgroup of the many-row kernel.
constexpr int fp8_tile_cols(bool gate_up) { return gate_up ? 128 : 256; }
// Token rows (in 16s) of one workgroup of the many-row kernel.
inline int fp8_tile_rows16(const Fp8Args& a, bool gate_up) { return 8; }

// Rows an expert has on average when every expert that can have rows has some.
inline int fp8_mean_rows(const Fp8Args& a) {
    const int groups = a.offsets ? (a.E < a.R ? a.E : a.R) : 1;
    return (a.R + groups - 1) / groups;
}

// Token rows (in 16s) of one workgroup of the few-row kernel.
inline int fp8_skinny_rows16(const Fp8Args& a) {
    const int m = fp8_mean_rows(a);
    return m <= 16 ? 1 : m <= 32 ? 2 : 4;
}

inline bool fp8_uses_skinny(const Fp8Args& a) { return fp8_mean_rows(a) <= (a.offsets ? 16 : 256); }

// Workgroups of a call's product launch; the entry points refuse more than a
// grid's 2^31 - 1.
inline long long fp8_blocks(const Fp8Args& a, bool gate_up) {
    if (fp8_uses_skinny(a)) return static_cast<long long>((a.N + 15) / 16) * row_items(a, 16 * fp8_skinny_rows16(a));
    const int cols = fp8_tile_cols(gate_up);
    return static_cast<long long>((a.N + cols - 1) / cols) * ((row_items(a, 16 * fp8_tile_rows16(a, gate_up)) + 7) / 8 * 8);
}

hipError_t launch_fp8_skinny(const Fp8Args& a, bool gate_up, hipStream_t st);
hipError_t launch_fp8_tile(const Fp8Args& a, bool gate_up, hipStream_t st);

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
