// FP8 products of few token rows (moe_gemm_fp8, moe_grouped_gemm_fp8 and
// moe_expert_gate_up_fp8 at decode, verify and small batches).
//
// out[m][n] = sum over steps s of 128 of as[m][s] * ws[n/128][s] * (a . w in
// the step).  Bound by the stream of the weights, each byte of which is read
// once per run of 16 token rows.  A workgroup computes 16 weight rows (gate
// and up: 16 of each) x 16 token rows; its waves split the steps, every wave
// accumulates its own in fp32 and the partial tiles are summed in LDS in wave
// order, so results do not depend on timing.
//
// The weights go from memory to the matrix operand: lane l reads 16-byte
// chunks l/16 and 4 + l/16 of row l%16's 128 bytes, so the two loads of a step
// consume 16 whole cache lines.  What keeps enough on its way is the number of
// waves (up to 32 a CU), not requests ahead in each: one row x 4096 x 4096 takes
// 5.4 us (2.7 of them a launch of any size), 25 experts of 4096 x 2048 with a
// row or two each 40 us, the weights at 5.3 TB/s; with two chunks of two steps
// held ahead, both built for one run, 6.9 beside 6.0 and 65 beside 40.
//
// Operands are bf16 (E4M3 converts exactly) on the 16x16x32 instruction: the
// fp8 instructions align their products before adding (1.5e-5 relative per
// step, measured), and the rate is of no concern here.  Weights are the A
// operand, so a lane's four outputs belong to one token and a step's two
// scales are one factor.  K is permuted inside a step, the same for weights
// and tokens: lane l takes chunks l/16 and 4 + l/16 of its row.
#include "fp8.hpp"
#include "kernels.hpp"

namespace qrmoe {

namespace {

__device__ __forceinline__ void to_operands(u32x4 c0, u32x4 c1, bf16x8 (&o)[4]) {
    o[0] = e4m3x8_to_bf16(c0[0], c0[1]);
    o[1] = e4m3x8_to_bf16(c0[2], c0[3]);
    o[2] = e4m3x8_to_bf16(c1[0], c1[1]);
    o[3] = e4m3x8_to_bf16(c1[2], c1[3]);
}

// KW: waves that split the steps.
template <int MATS, int KW>
__device__ __forceinline__ void few_body(const Fp8Args& a, int n_tiles, float* part) {
    const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n_tile = blockIdx.x % n_tiles, item = blockIdx.x / n_tiles, n0 = n_tile * 16;
    const RowItem it = row_item(a, item, 16, MATS == 1);
    if (it.e < 0) return;
    if (MATS == 1 && it.e == a.E) return zero_tile<16>(a, it, n0);
    const int S = ceil_div(a.K, kRun), NB = ceil_div(a.N, kRun);
    const int s_beg = S * wave / KW, s_end = S * (wave + 1) / KW;

    const uint8_t* wrow[MATS];
    Scalar* wscale[MATS];
#pragma unroll
    for (int m = 0; m < MATS; ++m) {
        wrow[m] = a.w[m] + (static_cast<size_t>(it.e) * a.N + min(n0 + col, a.N - 1)) * a.K;
        wscale[m] = scalar_ptr(a.w_scales[m] + (static_cast<size_t>(it.e) * NB + n0 / kRun) * S);
    }
    const int src = source_row(a, min(it.r0 + col, it.r1 - 1));
    const uint8_t* arow = a.a + src * a.a_stride;
    const float* ascale = a.a_scales + static_cast<size_t>(src) * S;
    f32x4 acc[MATS];
#pragma unroll
    for (int m = 0; m < MATS; ++m) acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    // chunk k of a row, zeros past K (a multiple of 32: a chunk is inside or not)
    auto chunk = [&](const uint8_t* row, int k) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(row + (k < a.K ? k : 0));
        return k < a.K ? v : u32x4{0u, 0u, 0u, 0u};
    };
#pragma unroll 2
    for (int s = s_beg; s < s_end; ++s) {
        const int k = s * kRun + 16 * g;
        u32x4 w[MATS][2];
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
            w[m][0] = chunk(wrow[m], k);
            w[m][1] = chunk(wrow[m], k + 64);
        }
        bf16x8 ao[4];
        to_operands(chunk(arow, k), chunk(arow, k + 64), ao);
        const float ts = ascale[s];
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
            bf16x8 wo[4];
            to_operands(w[m][0], w[m][1], wo);
            f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 4; ++j) p = mfma16x16x32(wo[j], ao[j], p);
            const float f = ts * wscale[m][s];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][i] = fmaf(p[i], f, acc[m][i]);
        }
    }

    // partial tile of matrix m: value [token col][weight row 4 g + i]
#pragma unroll
    for (int m = 0; m < MATS; ++m) *reinterpret_cast<f32x4*>(part + (wave * MATS + m) * 256 + col * 16 + 4 * g) = acc[m];
    __syncthreads();
    const int i = threadIdx.x;
    if (i < 256) {
        float v[MATS];
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
            v[m] = 0.f;
#pragma unroll
            for (int w = 0; w < KW; ++w) v[m] += part[(w * MATS + m) * 256 + i];
        }
        const int r = it.r0 + i / 16, n = n0 + i % 16;
        if (r < it.r1 && n < a.N) {
            if constexpr (MATS == 2) {
                store_hidden(a, r, n, silu_mul(v[0], v[1]));
            } else {
                const long long at = r * a.out_stride + n;
                if (a.out_f32) static_cast<float*>(a.out)[at] = v[0];
                else static_cast<uint16_t*>(a.out)[at] = f32_to_bf16_rne(v[0]);
            }
        }
    }
    if constexpr (MATS == 2) finish_run<16>(a, it, item, n_tile, n_tiles, reinterpret_cast<int*>(part + KW * MATS * 256));
}

template <int MATS, int KW>
__global__ __launch_bounds__(KW* kWave) void fp8_few_kernel(Fp8Args a, int n_tiles) {
    __shared__ __align__(16) float part[KW * MATS * 256 + 4];       // partial tiles, and a word of finish_run
    few_body<MATS, KW>(a, n_tiles, part);
}

}  // namespace

// Eight waves where each has three steps or more (32 steps, 1 x 4096 x 4096, in
// one run: eight 5.9 us, four 7.2; gate/up, 29 experts: 91, 95) or there is no more than
// one workgroup a CU (16 steps, 1 x 4096 x 2048: 4.3, 4.9); else four (16 steps,
// 23 experts of 4096 x 2048: 45, 40).
hipError_t launch_fp8_few(const Fp8Args& a, const Fp8Plan& p, bool gate_up, hipStream_t st) {
    const int blocks = static_cast<int>(p.blocks);
    const bool eight = ceil_div(a.K, kRun) >= 24 || static_cast<long long>(p.n_tiles) * p.products <= 256;
    if (gate_up && eight) fp8_few_kernel<2, 8><<<blocks, 8 * kWave, 0, st>>>(a, p.n_tiles);
    else if (gate_up) fp8_few_kernel<2, 4><<<blocks, 4 * kWave, 0, st>>>(a, p.n_tiles);
    else if (eight) fp8_few_kernel<1, 8><<<blocks, 8 * kWave, 0, st>>>(a, p.n_tiles);
    else fp8_few_kernel<1, 4><<<blocks, 4 * kWave, 0, st>>>(a, p.n_tiles);
    return hipGetLastError();
}

}  // namespace qrmoe
