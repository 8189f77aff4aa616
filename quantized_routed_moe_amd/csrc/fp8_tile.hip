// FP8 products of many token rows (moe_gemm_fp8, moe_grouped_gemm_fp8 and
// moe_expert_gate_up_fp8 at prefill sizes).
//
// out[m][n] = sum over steps s of 128 of as[m][s] * ws[n/128][s] * (a . w in
// the step): the products of a step run on the matrix cores from zero and
// one fp32 multiply-add per output and step adds them, scaled, to the
// accumulators.
//
// A workgroup of four waves computes 256 weight rows x 16*MT token rows; wave
// w owns 64 weight rows (gate/up: 32 gate rows and the same 32 up rows), so
// no two waves need the same weights and each wave loads its own straight
// from memory into the matrix operand, one step ahead.  The token rows are
// shared: they are staged in LDS, two buffers, swizzled so that the 16 rows
// of a fragment read start in distinct banks.
//
// FAST: operands stay E4M3 on the 16x16x128 fp8 instruction, whose internal
// alignment costs about 1.5e-5 relative per step (measured on normal values);
// used for bf16 results only.  Otherwise operands are converted to bf16
// (exact) and the products run on the 16x16x32 bf16 instruction at half the
// rate, with fp32 accuracy.
#include "fp8.hpp"
#include "kernels.hpp"

namespace qrmoe {

namespace {

constexpr int kTileN = 256;
constexpr int kTileThreads = 256;

template <bool FAST> constexpr int kRowBytes = FAST ? 128 : 256;

// LDS offset of 16-byte chunk c of token row r.  E4M3 rows of 128 bytes (8
// chunks): two rows span the 64 banks, so rows 2i and 2i+1 share a key; bf16
// rows of 256 bytes (16 chunks).
template <bool FAST>
__device__ __forceinline__ int swz(int r, int c) {
    if constexpr (FAST) return r * 128 + ((c ^ ((r >> 1) & 7)) << 4);
    else return r * 256 + ((c ^ (r & 15)) << 4);
}

__device__ __forceinline__ u32x4 load_chunk(const uint8_t* row, int k, int K) {
    const bool in = k < K;      // K is a multiple of 32: a chunk is inside or outside
    const u32x4 v = *reinterpret_cast<const u32x4*>(row + (in ? k : 0));
    return in ? v : u32x4{0u, 0u, 0u, 0u};
}

template <bool FAST> struct WOp;
template <> struct WOp<true> {
    i32x8 v;
    __device__ __forceinline__ void set(u32x4 lo, u32x4 hi) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = static_cast<int>(lo[i]);
            v[4 + i] = static_cast<int>(hi[i]);
        }
    }
};
template <> struct WOp<false> {
    bf16x8 v[4];
    __device__ __forceinline__ void set(u32x4 lo, u32x4 hi) {
        v[0] = e4m3x8_to_bf16(lo[0], lo[1]);
        v[1] = e4m3x8_to_bf16(lo[2], lo[3]);
        v[2] = e4m3x8_to_bf16(hi[0], hi[1]);
        v[3] = e4m3x8_to_bf16(hi[2], hi[3]);
    }
};

__device__ __forceinline__ f32x4 step_product(const WOp<true>& w, const WOp<true>& t) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, t.v, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 step_product(const WOp<false>& w, const WOp<false>& t) {
    f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j) p = mfma16x16x32(w.v[j], t.v[j], p);
    return p;
}

// GU: gate/up with SwiGLU and E4M3 output, 128 columns of act per workgroup.
template <int MT, bool GU, bool FAST>
__global__ __launch_bounds__(kTileThreads, 2) void fp8_tile_kernel(Fp8Args a, int n_tiles) {
    constexpr int kRows = 16 * MT;
    constexpr int kCols = GU ? kTileN / 2 : kTileN;     // output columns
    constexpr int kChunks = kRows * 8 / kTileThreads;   // 16-byte token chunks a thread stages per step
    __shared__ __align__(16) uint8_t tok[2][kRows * kRowBytes<FAST>];
    __shared__ float tscale[2][kRows];
    __shared__ float rowmax[GU ? 4 : 1][GU ? kRows : 1];

    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, col = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n_tile = blockIdx.x % n_tiles, item = blockIdx.x / n_tiles;
    const int n0 = n_tile * kCols;
    if constexpr (!GU)
        if (a.offsets && item == 0) zero_rows_past_end(a, n0, min(n0 + kCols, a.N));
    const RowItem it = row_item(a, item, kRows);
    if (it.e < 0) return;
    const int S = ceil_div(a.K, kRun), NB = ceil_div(a.N, kRun);

    // this wave's four 16-row weight fragments
    const uint8_t* wrow[4];
    const float* wscale[4];
    int wn[4];                                          // first output column of the fragment
#pragma unroll
    for (int f = 0; f < 4; ++f) {
        const int m = GU ? f >> 1 : 0;
        wn[f] = GU ? n0 + 32 * wave + 16 * (f & 1) : n0 + 64 * wave + 16 * f;
        const int row = min(wn[f] + col, a.N - 1);
        wrow[f] = a.w[m] + (static_cast<size_t>(it.e) * a.N + row) * a.K;
        wscale[f] = a.w_scales[m] + (static_cast<size_t>(it.e) * NB + min(wn[f], a.N - 1) / kRun) * S;
    }
    // the token chunks this thread stages: chunk tid%8 of rows tid/8 + 32 i
    const uint8_t* trow[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
        trow[i] = a.a + source_row(a, min(it.r0 + tid / 8 + 32 * i, it.r1 - 1)) * a.a_stride;
    const float* trow_scale = a.a_scales + static_cast<size_t>(source_row(a, min(it.r0 + min(tid, kRows - 1), it.r1 - 1))) * S;

    u32x4 wnext[4][2], tnext[kChunks];
    float snext;
    auto fetch = [&](int s) {
#pragma unroll
        for (int f = 0; f < 4; ++f)
#pragma unroll
            for (int h = 0; h < 2; ++h) wnext[f][h] = load_chunk(wrow[f], s * kRun + 64 * h + 16 * g, a.K);
#pragma unroll
        for (int i = 0; i < kChunks; ++i) tnext[i] = load_chunk(trow[i], s * kRun + 16 * (tid & 7), a.K);
        snext = trow_scale[s];
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int r = tid / 8 + 32 * i, c = tid & 7;
            if constexpr (FAST) {
                *reinterpret_cast<u32x4*>(&tok[buf][swz<true>(r, c)]) = tnext[i];
            } else {
                *reinterpret_cast<bf16x8*>(&tok[buf][swz<false>(r, 2 * c)]) = e4m3x8_to_bf16(tnext[i][0], tnext[i][1]);
                *reinterpret_cast<bf16x8*>(&tok[buf][swz<false>(r, 2 * c + 1)]) = e4m3x8_to_bf16(tnext[i][2], tnext[i][3]);
            }
        }
        if (tid < kRows) tscale[buf][tid] = snext;
    };

    f32x4 acc[4][MT];
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[f][t] = f32x4{0.f, 0.f, 0.f, 0.f};

    fetch(0);
    stage(0);
    for (int s = 0; s < S; ++s) {
        WOp<FAST> wo[4];
        float ws[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            wo[f].set(wnext[f][0], wnext[f][1]);
            ws[f] = wscale[f][s];
        }
        __syncthreads();
        if (s + 1 < S) fetch(s + 1);
        const uint8_t* buf = tok[s & 1];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int r = 16 * t + col;
            WOp<FAST> to;
            if constexpr (FAST) {
                to.set(*reinterpret_cast<const u32x4*>(&buf[swz<true>(r, g)]),
                       *reinterpret_cast<const u32x4*>(&buf[swz<true>(r, 4 + g)]));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    to.v[j] = *reinterpret_cast<const bf16x8*>(&buf[swz<false>(r, (j >> 1) * 8 + 2 * g + (j & 1))]);
            }
            const float ts = tscale[s & 1][r];
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const f32x4 p = step_product(wo[f], to);
                const float m = ts * ws[f];
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[f][t][i] = fmaf(p[i], m, acc[f][t][i]);
            }
        }
        if (s + 1 < S) stage((s + 1) & 1);
    }

    if constexpr (!GU) {
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int r = it.r0 + 16 * t + col;
            if (r >= it.r1) continue;
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const int n = wn[f] + 4 * g;
                const long long at = r * a.out_stride + n;
                const f32x4 v = acc[f][t];
                if (a.out_vec && n + 4 <= a.N) {
                    if constexpr (FAST)
                        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + at) =
                            u32x2{f32_to_bf16_rne(v[0]) | static_cast<uint32_t>(f32_to_bf16_rne(v[1])) << 16,
                                  f32_to_bf16_rne(v[2]) | static_cast<uint32_t>(f32_to_bf16_rne(v[3])) << 16};
                    else *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + at) = v;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (n + i < a.N) {
                            if constexpr (FAST) static_cast<uint16_t*>(a.out)[at + i] = f32_to_bf16_rne(v[i]);
                            else static_cast<float*>(a.out)[at + i] = v[i];
                        }
                }
            }
        }
    } else {
        // v = silu(g) u in place of the gate accumulators; a run's 128
        // columns are the workgroup's, 8 per lane and token
        const bool in = wn[0] < a.N;        // f is a multiple of 32: a wave's columns are inside or outside
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            float m = 0.f;
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[f][t][i] = in ? silu_mul(acc[f][t][i], acc[2 + f][t][i]) : 0.f;
                    m = fmaxf(m, fabsf(acc[f][t][i]));
                }
            m = fmaxf(m, __shfl_xor(m, 16));
            m = fmaxf(m, __shfl_xor(m, 32));
            if (g == 0) rowmax[wave][16 * t + col] = m;
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int rt = 16 * t + col, r = it.r0 + rt;
            if (r >= it.r1) continue;
            const float s = run_scale(fmaxf(fmaxf(rowmax[0][rt], rowmax[1][rt]), fmaxf(rowmax[2][rt], rowmax[3][rt])));
            if (wave == 0 && g == 0) a.act_scales[static_cast<size_t>(r) * NB + n_tile] = s;
            if (!in) continue;
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const f32x4 v = acc[f][t];
                *reinterpret_cast<uint32_t*>(a.act + static_cast<size_t>(r) * a.N + wn[f] + 4 * g) =
                    e4m3x4_rne(v[0] / s, v[1] / s, v[2] / s, v[3] / s);
            }
        }
    }
}

}  // namespace

hipError_t launch_fp8_tile(const Fp8Args& a, bool gate_up, hipStream_t st) {
    const int n_tiles = ceil_div(a.N, fp8_tile_cols(gate_up));
    const int blocks = static_cast<int>(fp8_blocks(a, gate_up));
    if (gate_up) fp8_tile_kernel<4, true, false><<<blocks, kTileThreads, 0, st>>>(a, n_tiles);
    else if (a.out_f32) fp8_tile_kernel<4, false, false><<<blocks, kTileThreads, 0, st>>>(a, n_tiles);
    else fp8_tile_kernel<8, false, true><<<blocks, kTileThreads, 0, st>>>(a, n_tiles);
    return hipGetLastError();
}

}  // namespace qrmoe
