// FP8 products of few token rows (moe_gemm_fp8, moe_grouped_gemm_fp8 and
// moe_expert_gate_up_fp8 at decode, verify and small batches).
//
// out[m][n] = sum over steps s of 128 of as[m][s] * ws[n/128][s] * (a . w in
// the step).  Bound by the stream of the weights, each byte of which is read
// once per run of token rows.  A workgroup computes 16 weight rows (gate and
// up: 16 of each) x 16*MT token rows; its KW waves split the steps, every
// wave accumulates its steps in fp32 and the partial tiles are summed in LDS
// in wave order, so results do not depend on timing.
//
// The weights go from memory to the matrix operand: lane l reads 16-byte
// chunks l/16 and 4 + l/16 of row l%16's 128 bytes, so the two loads of a
// step consume 16 whole cache lines.  K is permuted inside the step by that
// choice, the same for the token rows.  Operands are bf16 (E4M3 converts
// exactly) on the 16x16x32 instruction: the fp8 instructions align their
// products before adding (1.5e-5 relative per step, measured), and the rate
// is of no concern here.  Weights are the A operand, so a lane's four
// outputs belong to one token and a step's two scales are one factor.
#include "fp8.hpp"
#include "kernels.hpp"

namespace qrmoe {

namespace {

// Chunks l/16 and 4 + l/16 of step s of a row (zeros past K).
struct Chunk2 {
    u32x4 c[2];
};

__device__ __forceinline__ Chunk2 load_step(const uint8_t* row, int s, int K, int g) {
    Chunk2 r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int k = s * kRun + 64 * h + 16 * g;
        const bool in = k < K;      // K is a multiple of 32: a chunk is inside or outside
        const u32x4 v = *reinterpret_cast<const u32x4*>(row + (in ? k : 0));
        r.c[h] = in ? v : u32x4{0u, 0u, 0u, 0u};
    }
    return r;
}

__device__ __forceinline__ void to_operands(const Chunk2& c, bf16x8 (&o)[4]) {
    o[0] = e4m3x8_to_bf16(c.c[0][0], c.c[0][1]);
    o[1] = e4m3x8_to_bf16(c.c[0][2], c.c[0][3]);
    o[2] = e4m3x8_to_bf16(c.c[1][0], c.c[1][1]);
    o[3] = e4m3x8_to_bf16(c.c[1][2], c.c[1][3]);
}

constexpr int kSkinnyWaves = 8;

template <int MT, int MATS>
__global__ __launch_bounds__(kSkinnyWaves* kWave) void fp8_skinny_kernel(Fp8Args a, int n_tiles) {
    constexpr int KW = kSkinnyWaves;
    constexpr int kOut = MATS * MT * 256;         // partial sums of a wave
    __shared__ float part[KW][kOut];
    const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = (blockIdx.x % n_tiles) * 16, item = blockIdx.x / n_tiles;
    if (a.offsets && !a.hidden && item == 0) zero_rows_past_end(a, n0, min(n0 + 16, a.N));
    const RowItem it = row_item(a, item, 16 * MT);
    if (it.e < 0) return;
    const int S = ceil_div(a.K, kRun), NB = ceil_div(a.N, kRun);
    const int s_beg = S * wave / KW, s_end = S * (wave + 1) / KW;

    const uint8_t* wrow[MATS];
    const float* wscale[MATS];
#pragma unroll
    for (int m = 0; m < MATS; ++m) {
        wrow[m] = a.w[m] + (static_cast<size_t>(it.e) * a.N + min(n0 + col, a.N - 1)) * a.K;
        wscale[m] = a.w_scales[m] + (static_cast<size_t>(it.e) * NB + n0 / kRun) * S;
    }
    const uint8_t* arow[MT];
    const float* ascale[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int src = source_row(a, min(it.r0 + 16 * t + col, it.r1 - 1));
        arow[t] = a.a + src * a.a_stride;
        ascale[t] = a.a_scales + static_cast<size_t>(src) * S;
    }
    f32x4 acc[MATS][MT];
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[m][t] = f32x4{0.f, 0.f, 0.f, 0.f};

#pragma unroll 4
    for (int s = s_beg; s < s_end; ++s) {
        Chunk2 wc[MATS];
#pragma unroll
        for (int m = 0; m < MATS; ++m) wc[m] = load_step(wrow[m], s, a.K, g);
        bf16x8 wo[MATS][4];
#pragma unroll
        for (int m = 0; m < MATS; ++m) to_operands(wc[m], wo[m]);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            bf16x8 ao[4];
            to_operands(load_step(arow[t], s, a.K, g), ao);
            const float as = ascale[t][s];
#pragma unroll
            for (int m = 0; m < MATS; ++m) {
                f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < 4; ++j) p = mfma16x16x32(wo[m][j], ao[j], p);
                const float f = as * wscale[m][s];
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][t][i] = fmaf(p[i], f, acc[m][t][i]);
            }
        }
    }
    // partial tile (m, t): value [token col][weight row 4g + i]
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int t = 0; t < MT; ++t)
            *reinterpret_cast<f32x4*>(&part[wave][(m * MT + t) * 256 + col * 16 + 4 * g]) = acc[m][t];
    __syncthreads();
    for (int i = threadIdx.x; i < MT * 256; i += KW * kWave) {
        float v[MATS];
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
            v[m] = 0.f;
#pragma unroll
            for (int w = 0; w < KW; ++w) v[m] += part[w][m * MT * 256 + i];
        }
        const int r = it.r0 + i / 16, n = n0 + i % 16;
        if (r >= it.r1 || n >= a.N) continue;
        if constexpr (MATS == 2) {
            a.hidden[static_cast<size_t>(r) * a.N + n] = silu_mul(v[0], v[1]);
        } else {
            const long long at = r * a.out_stride + n;
            if (a.out_f32) static_cast<float*>(a.out)[at] = v[0];
            else static_cast<uint16_t*>(a.out)[at] = f32_to_bf16_rne(v[0]);
        }
    }
}

// hidden -> E4M3 codes and scales, one wave per run of 128 values: two
// values per lane.
__global__ __launch_bounds__(256) void run_quant_kernel(Fp8Args a, int NB) {
    const int end = min(max(a.offsets[a.E], 0), a.R);
    const int lane = threadIdx.x & 63;
    const int wave = blockIdx.x * 4 + (threadIdx.x >> 6);
    const int r = wave / NB, b = wave % NB;
    if (r >= end) return;
    const int n = b * kRun + 2 * lane;
    const bool live = n < a.N;
    float v0 = 0.f, v1 = 0.f;
    if (live) {
        const f32x2 v = *reinterpret_cast<const f32x2*>(a.hidden + static_cast<size_t>(r) * a.N + n);
        v0 = v[0];
        v1 = v[1];
    }
    float m = fmaxf(fabsf(v0), fabsf(v1));
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
    const float s = run_scale(m);
    if (live)
        *reinterpret_cast<uint16_t*>(a.act + static_cast<size_t>(r) * a.N + n) =
            static_cast<uint16_t>(e4m3x4_rne(v0 / s, v1 / s, 0.f, 0.f));
    if (lane == 0) a.act_scales[static_cast<size_t>(r) * NB + b] = s;
}

template <int MATS>
hipError_t launch(const Fp8Args& a, hipStream_t st) {
    const int n_tiles = ceil_div(a.N, 16);
    const int threads = kSkinnyWaves * kWave;
    const int blocks = static_cast<int>(fp8_blocks(a, MATS == 2));
    switch (fp8_skinny_rows16(a)) {
        case 1: fp8_skinny_kernel<1, MATS><<<blocks, threads, 0, st>>>(a, n_tiles); break;
        case 2: fp8_skinny_kernel<2, MATS><<<blocks, threads, 0, st>>>(a, n_tiles); break;
        default: fp8_skinny_kernel<4, MATS><<<blocks, threads, 0, st>>>(a, n_tiles); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_skinny(const Fp8Args& a, bool gate_up, hipStream_t st) {
    if (!gate_up) return launch<1>(a, st);
    const hipError_t e = launch<2>(a, st);
    if (e != hipSuccess) return e;
    const int NB = ceil_div(a.N, kRun);
    run_quant_kernel<<<ceil_div(a.R * NB, 4), 256, 0, st>>>(a, NB);
    return hipGetLastError();
}

}  // namespace qrmoe
