// FP8 products of many token rows (moe_gemm_fp8, moe_grouped_gemm_fp8 and
// moe_expert_gate_up_fp8 at prefill sizes).
//
// out[m][n] = sum over steps s of 128 of as[m][s] * ws[n/128][s] * (a . w in
// the step): the products of a step run on the matrix cores from zero and
// one fp32 multiply-add per output and step adds them, scaled, to the
// accumulators.
//
// A workgroup computes 256 weight rows (gate/up: 128 gate rows and the same
// 128 up rows) x up to 128 token rows of one expert with eight waves, or, where
// that would leave most of the chip idle, 64 (32 and 32) x up to 64 with four.
// Both operands go from memory to LDS as they are, by direct copies of 16 bytes
// a lane, into a ring of stages of one step each: eight neighbouring lanes take
// one row's 128 bytes, whole cache lines.  (Loading the matrix operands
// straight into registers, lane = row, asks for 16 bytes of another line in
// every lane; that path stopped at 6 TB/s from the caches, whatever the
// prefetch distance.)  The 16-byte chunks of a row are stored XOR-swizzled by
// (row / 2) mod 8, so the 16 rows of a fragment read lie in distinct banks.
//
// The waves of the large tile split it by its live rows: 4 x 2 waves of 64
// weight rows x 64 token rows above 64 rows, else 8 waves of 32 weight rows x
// all token rows (64, 32 or 16), whose smaller stages leave room for a deeper
// ring.
//
// Fragments are converted to bf16 (exact) for the 16x16x32 bf16 instruction.
// The fp8 instructions would take the codes as they are at twice the rate
// (16x16x128), but they cut a step's products off 16 bits below its largest,
// which is not a sum in fp32 where large products cancel: 2048 x 4096 x 4096
// with a bf16 result, in one run, takes 72 us this way and 47 that way.
#include <type_traits>

#include "fp8.hpp"
#include "kernels.hpp"

namespace qrmoe {

namespace {

// A workgroup's tile: TN weight rows x up to TM token rows.
template <int TN> struct Tile;
template <> struct Tile<256> {
    static constexpr int waves = 8, most_rows = 128, lds = 149504;
};
template <> struct Tile<64> {
    static constexpr int waves = 4, most_rows = 64, lds = 67584;
};

// WM: waves along the token rows, TT: 16-row token tiles of a wave.
template <int TN, int WM, int TT> struct Shape {
    static constexpr int waves = Tile<TN>::waves;
    static constexpr int rows = 16 * TT * WM;       // token rows of a stage
    static constexpr int wn = waves / WM;           // waves along the weight rows
    static constexpr int frags = TN / 16 / wn;      // 16-row weight fragments of a wave
    static constexpr int wbytes = TN * kRun;
    static constexpr int stage = wbytes + rows * kRun + 512;      // weights, tokens, token scales
    static constexpr int fit = Tile<TN>::lds / stage;
    static constexpr int ring = fit > 4 ? 4 : fit;
    // copies of a wave per stage: weights, tokens (8 rows each), token scales
    static constexpr int share = rows / waves;      // token rows a wave copies
    static constexpr int wcopies = TN / waves / 8, tcopies = share > 8 ? share / 8 : 1;
    static constexpr int loads = wcopies + tcopies + 1;
    static_assert(ring >= 3 && rows <= Tile<TN>::most_rows, "stage ring");
};

// At most r (<= R) stages of L copies each are still in flight.
template <int L, int R>
__device__ __forceinline__ void wait_stages(int r) {
    if constexpr (R == 0) {
        wait_vmcnt<0>();
    } else {
        if (r >= R) wait_vmcnt<R * L>();
        else wait_stages<L, R - 1>(r);
    }
}

// Every wave has finished its LDS reads and the copies it waited for; no
// LDS access moves across.
__device__ __forceinline__ void stage_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A fragment's operand: chunks l/16 and 4 + l/16 of row l%16 (K is permuted
// inside the step by that choice, the same for weights and tokens).
struct Operand {
    bf16x8 v[4];
    __device__ __forceinline__ void set(u32x4 lo, u32x4 hi) {
        v[0] = e4m3x8_to_bf16(lo[0], lo[1]);
        v[1] = e4m3x8_to_bf16(lo[2], lo[3]);
        v[2] = e4m3x8_to_bf16(hi[0], hi[1]);
        v[3] = e4m3x8_to_bf16(hi[2], hi[3]);
    }
};

// The step's products of a wave's weight fragments and one token tile.
template <int F>
__device__ __forceinline__ void step_products(const Operand (&w)[F], const Operand& t, f32x4 (&p)[F]) {
#pragma unroll
    for (int f = 0; f < F; ++f) p[f] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int f = 0; f < F; ++f) p[f] = mfma16x16x32(w[f].v[j], t.v[j], p[f]);
}

// One workgroup's product.  GU: gate/up with SwiGLU and E4M3 output; else
// BF: bf16 output, not fp32.
template <int TN, int WM, int TT, bool GU, bool BF>
__device__ __forceinline__ void tile_body(const Fp8Args& a, const RowItem& it, int n_tile, uint8_t* lds) {
    using H = Shape<TN, WM, TT>;
    constexpr int F = H::frags, FG = F / 2, NST = H::ring, SB = H::stage, L = H::loads;
    constexpr int kCols = GU ? TN / 2 : TN;             // output columns
    constexpr bool kRuns = GU && kCols == kRun;         // whole runs of 128: E4M3 from here
    constexpr int kWBytes = H::wbytes;
    constexpr int kMats = GU ? 2 : 1;

    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, col = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave & (H::wn - 1), wm = wave / H::wn;
    const int n0 = n_tile * kCols;
    const int S = ceil_div(a.K, kRun), NB = ceil_div(a.N, kRun);
    const int full = a.K / kRun;                        // whole steps
    // ---- copies: the wave's share of the tile's weight rows, 8 rows each
    // (gate/up: the first half of the waves gate, the second up), position lane%8 of the row in LDS holding chunk
    // (lane%8) ^ (row/2)%8
    constexpr int kShareW = 8 * H::wcopies;             // weight rows of a wave
    const int mat = GU ? wave / (H::waves / 2) : 0;
    const __amdgpu_buffer_rsrc_t wbuf = buffer_of(a.w[mat] + (static_cast<size_t>(it.e) * a.N + n0) * a.K);
    const int chunk0 = (lane & 7) ^ (lane >> 4);        // rows of even 8 i; of odd 8 i: chunk0 ^ 4
    int woff[H::wcopies];
#pragma unroll
    for (int i = 0; i < H::wcopies; ++i) {
        const int row = kShareW * (GU ? wave % (H::waves / 2) : wave) + 8 * i + (lane >> 3);
        woff[i] = min(row, a.N - 1 - n0) * a.K + 16 * (chunk0 ^ (4 * (i & 1)));     // at most 256 * 2^22
    }
    // token rows: the wave's share of the stage's rows, tcopies times 8 (64
    // rows or more) or fewer rows in the low lanes
    constexpr int kShare = H::share;
    const uint8_t* tsrc[H::tcopies];
#pragma unroll
    for (int i = 0; i < H::tcopies; ++i) {
        const int row = kShare * wave + 8 * i + (lane >> 3);
        tsrc[i] = a.a + source_row(a, min(it.r0 + row, it.r1 - 1)) * a.a_stride + 16 * ((lane & 7) ^ ((row >> 1) & 7));
    }
    const float* ssrc = a.a_scales + static_cast<size_t>(source_row(a, min(it.r0 + kShare * wave + (lane & 15), it.r1 - 1))) * S;
    auto issue = [&](int s) {
        uint8_t* base = lds + (s % NST) * SB;
        // the partial step: a chunk past K is read from the step's start (and
        // cleared when it is used)
        const int part = s == full ? -1 : 0;
#pragma unroll
        for (int c = 0; c < H::wcopies; ++c) {
            const int k = 16 * (chunk0 ^ (4 * (c & 1)));
            const int back = (full * kRun + k < a.K ? 0 : k) & part;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(wbuf, (lds_void*)(base + (kShareW * wave + 8 * c) * kRun), 16, woff[c] - back,
                                                     s * kRun, 0, 0);
        }
#pragma unroll
        for (int c = 0; c < H::tcopies; ++c) {
            const int k = 16 * ((lane & 7) ^ (((kShare * wave + 8 * c + (lane >> 3)) >> 1) & 7));
            const int back = (full * kRun + k < a.K ? 0 : k) & part;
            if (kShare >= 8 || lane < 8 * kShare)
                __builtin_amdgcn_global_load_lds(tsrc[c] + (s * kRun - back), (lds_void*)(base + kWBytes + (kShare * wave + 8 * c) * kRun),
                                                 16, 0, 0);
        }
        if (lane < kShare)
            __builtin_amdgcn_global_load_lds(ssrc + s, (lds_void*)(base + kWBytes + H::rows * kRun + 4 * kShare * wave), 4, 0, 0);
    };

    // ---- this wave's fragments: weight rows of the tile and output columns
    int wrow[F], wcol[F];
    Scalar* wscale[kMats];
#pragma unroll
    for (int f = 0; f < F; ++f) {
        const int c = GU ? 16 * FG * wn + 16 * (f % FG) : 16 * F * wn + 16 * f;
        wrow[f] = GU ? kCols * (f / FG) + c : c;
        wcol[f] = n0 + c;
    }
#pragma unroll
    for (int m = 0; m < kMats; ++m)      // a wave's columns share a block of 128
        wscale[m] = scalar_ptr(a.w_scales[m] + (static_cast<size_t>(it.e) * NB + min(wcol[0], a.N - 1) / kRun) * S);
    // chunk l/16 of row l%16; chunk 4 + l/16 is at the offset ^ 64
    const int frag = col * kRun + ((g ^ (col >> 1)) << 4);

    f32x4 acc[F][TT];
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[f][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    float ws[kMats];
    auto load_ws = [&](int s) {
#pragma unroll
        for (int m = 0; m < kMats; ++m) ws[m] = wscale[m][s];
    };

    auto multiply = [&](int i, auto partial) {
        const uint8_t* base = lds + (i % NST) * SB;
        const uint8_t* lo = base + frag;
        const uint8_t* hi = base + (frag ^ 64);
        const uint8_t* tlo = lo + kWBytes + 16 * TT * wm * kRun;
        const uint8_t* thi = hi + kWBytes + 16 * TT * wm * kRun;
        const float* ts = reinterpret_cast<const float*>(base + kWBytes + H::rows * kRun) + 16 * TT * wm + col;
        auto operand = [&](Operand& o, const uint8_t* l, const uint8_t* h) {
            u32x4 c0 = *reinterpret_cast<const u32x4*>(l), c1 = *reinterpret_cast<const u32x4*>(h);
            if constexpr (partial) {
                if (full * kRun + 16 * g >= a.K) c0 = u32x4{0u, 0u, 0u, 0u};
                if (full * kRun + 64 + 16 * g >= a.K) c1 = u32x4{0u, 0u, 0u, 0u};
            }
            o.set(c0, c1);
        };
        float w[kMats];
#pragma unroll
        for (int m = 0; m < kMats; ++m) w[m] = ws[m];
        Operand wo[F];
#pragma unroll
        for (int f = 0; f < F; ++f) operand(wo[f], lo + wrow[f] * kRun, hi + wrow[f] * kRun);
        if (!partial) load_ws(min(i + 1, S - 1));
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            Operand to;
            operand(to, tlo + 16 * t * kRun, thi + 16 * t * kRun);
            f32x4 p[F];
            step_products(wo, to, p);
            const float s = ts[16 * t];
#pragma unroll
            for (int f = 0; f < F; ++f) {
                const float m = s * w[GU ? f / FG : 0];
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[f][t][q] = fmaf(p[f][q], m, acc[f][t][q]);
            }
        }
    };

    load_ws(0);
    for (int i = 0; i < NST - 1 && i < S; ++i) issue(i);
    // Step i: its copies have arrived (all but the younger stages'), every
    // wave is past step i - 1, whose buffer stage i + NST - 1 then takes.
    auto begin = [&](int i) {
        const int younger = min(S - 1, i + NST - 2) - i;
        if (younger == NST - 2) wait_vmcnt<L * (NST - 2)>();
        else wait_stages<L, NST - 2>(younger);
        stage_barrier();
        if (i + NST - 1 < S) issue(i + NST - 1);
        __builtin_amdgcn_sched_barrier(0);
    };
    for (int i = 0; i < full; ++i) {
        begin(i);
        multiply(i, std::false_type{});
    }
    if (full < S) {
        begin(full);
        multiply(full, std::true_type{});
    }

    if constexpr (!GU) {
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const int r = it.r0 + 16 * (TT * wm + t) + col;
            if (r >= it.r1) continue;
#pragma unroll
            for (int f = 0; f < F; ++f) {
                const int n = wcol[f] + 4 * g;
                const long long at = r * a.out_stride + n;
                const f32x4 v = acc[f][t];
                if (a.out_vec && n + 4 <= a.N) {
                    if constexpr (BF)
                        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + at) =
                            u32x2{f32_to_bf16_rne(v[0]) | static_cast<uint32_t>(f32_to_bf16_rne(v[1])) << 16,
                                  f32_to_bf16_rne(v[2]) | static_cast<uint32_t>(f32_to_bf16_rne(v[3])) << 16};
                    else *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + at) = v;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (n + i < a.N) {
                            if constexpr (BF) static_cast<uint16_t*>(a.out)[at + i] = f32_to_bf16_rne(v[i]);
                            else static_cast<float*>(a.out)[at + i] = v[i];
                        }
                }
            }
        }
    } else if constexpr (!kRuns) {
        // less than a run of columns: through the workspace (finish_run)
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const int r = it.r0 + 16 * (TT * wm + t) + col;
#pragma unroll
            for (int f = 0; f < FG; ++f)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (r < it.r1 && wcol[f] < a.N)
                        store_hidden(a, r, wcol[f] + 4 * g + i, silu_mul(acc[f][t][i], acc[FG + f][t][i]));
        }
    } else {
        // v = silu(g) u in place of the gate accumulators; a run's 128
        // columns are the workgroup's, 4 FG per lane and token
        float* rowmax = reinterpret_cast<float*>(lds);
        __syncthreads();
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            float m = 0.f;
#pragma unroll
            for (int f = 0; f < FG; ++f)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // f is a multiple of 32, so a fragment is inside or outside
                    acc[f][t][i] = wcol[f] < a.N ? silu_mul(acc[f][t][i], acc[FG + f][t][i]) : 0.f;
                    m = fmaxf(m, fabsf(acc[f][t][i]));
                }
            m = fmaxf(m, __shfl_xor(m, 16));
            m = fmaxf(m, __shfl_xor(m, 32));
            if (g == 0) rowmax[wn * H::rows + 16 * (TT * wm + t) + col] = m;
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const int rt = 16 * (TT * wm + t) + col, r = it.r0 + rt;
            if (r >= it.r1) continue;
            float m = rowmax[rt];
#pragma unroll
            for (int w = 1; w < H::wn; ++w) m = fmaxf(m, rowmax[w * H::rows + rt]);
            const float s = run_scale(m);
            if (wn == 0 && g == 0) a.act_scales[static_cast<size_t>(r) * NB + n_tile] = s;
#pragma unroll
            for (int f = 0; f < FG; ++f) {
                const f32x4 v = acc[f][t];
                if (wcol[f] < a.N)
                    *reinterpret_cast<uint32_t*>(a.act + static_cast<size_t>(r) * a.N + wcol[f] + 4 * g) =
                        e4m3x4_rne(v[0] / s, v[1] / s, v[2] / s, v[3] / s);
            }
        }
    }
}

template <int TN, bool GU, bool BF>
__global__ __launch_bounds__(Tile<TN>::waves* kWave, 2) void fp8_tile_kernel(Fp8Args a, int n_tiles, int group_bits, int items) {
    __shared__ __align__(256) uint8_t lds[Tile<TN>::lds];
    // Workgroup ids go round the 8 XCDs.  An XCD takes one of 2^group_bits groups
    // of column tiles (as even as they come, the grid has room for the largest)
    // and every (8 >> group_bits)-th item: its workgroups share both weight tiles
    // and token rows in its L2.  (One group instead of four, us: 256 x
    // 4096 x 4096 in fp32 21.7 -> 29.0; 8 experts of 4096 x 2048, T = 256, down
    // 26.2 -> 32.1, T = 2048 gate/up 183 -> 201; eight groups as four.)
    const int xcd = blockIdx.x % 8, at = blockIdx.x / 8, groups = 1 << group_bits, group = xcd % groups;
    const int per = (n_tiles + groups - 1) >> group_bits;
    const int n_tile = (group * n_tiles >> group_bits) + at % per;      // n_tiles <= 2^24
    const int item = at / per * (8 >> group_bits) + (xcd >> group_bits);
    if (n_tile >= (group + 1) * n_tiles >> group_bits) return;
    // offsets that overlap could make an item of the rounded-up grid's rest;
    // the workspace is sized for `items`
    if (item >= items) return;
    const RowItem it = row_item(a, item, Tile<TN>::most_rows, !GU);
    if (it.e < 0) return;
    if (!GU && it.e == a.E) return zero_tile<TN>(a, it, n_tile * TN);
    const int rows = __builtin_amdgcn_readfirstlane(it.r1 - it.r0);
    if constexpr (TN == 256) {
        if (rows > 64) tile_body<TN, 2, 4, GU, BF>(a, it, n_tile, lds);
        else if (rows > 32) tile_body<TN, 1, 4, GU, BF>(a, it, n_tile, lds);
        else if (rows > 16) tile_body<TN, 1, 2, GU, BF>(a, it, n_tile, lds);
        else tile_body<TN, 1, 1, GU, BF>(a, it, n_tile, lds);
    } else {
        if (rows > 32) tile_body<TN, 2, 2, GU, BF>(a, it, n_tile, lds);
        else tile_body<TN, 2, 1, GU, BF>(a, it, n_tile, lds);
        if constexpr (GU) {
            __syncthreads();
            finish_run<TN / 2>(a, it, item, n_tile, n_tiles, reinterpret_cast<int*>(lds));
        }
    }
}

template <int TN>
void launch(const Fp8Args& a, const Fp8Plan& p, bool gate_up, hipStream_t st) {
    const int threads = Tile<TN>::waves * kWave, blocks = static_cast<int>(p.blocks);
    if (gate_up) fp8_tile_kernel<TN, true, false><<<blocks, threads, 0, st>>>(a, p.n_tiles, p.group_bits, p.items);
    else if (a.out_f32) fp8_tile_kernel<TN, false, false><<<blocks, threads, 0, st>>>(a, p.n_tiles, p.group_bits, p.items);
    else fp8_tile_kernel<TN, false, true><<<blocks, threads, 0, st>>>(a, p.n_tiles, p.group_bits, p.items);
}

}  // namespace

hipError_t launch_fp8_tile(const Fp8Args& a, const Fp8Plan& p, bool gate_up, hipStream_t st) {
    if (p.path == Fp8Path::kMany) launch<256>(a, p, gate_up, st);
    else launch<64>(a, p, gate_up, st);
    return hipGetLastError();
}

}  // namespace qrmoe
