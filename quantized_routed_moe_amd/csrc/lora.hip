// Low-rank adapters of many requests beside a shared projection (moe_lora_add):
// v = a[g] x for every token with an adapter g, then out = base + scales[g] b[g] v.
//
// Few operations a byte: bound by HBM (x, the active adapters, base and out),
// with few tokens by launches and latency.  Two launches.  The shrink takes
// runs of 16 tokens of one adapter, 16 to 64 ranks and a part of K; its waves
// split the part, and their sums meet in LDS in wave order.  The expand takes a
// run of up to 64 tokens and 256 columns and adds the parts of v in order, so
// nothing depends on timing.
//
// Both are 16x16x32 bf16 products with the weights as operand A, so a lane's
// four results are neighbouring ranks or columns of one token.  bf16 products
// are exact in fp32.  v is fp32: for the expand it is split into three bf16
// parts that hold its 24 bits, and three products are added (the matrix work is a
// few per cent of the time that base and out take).
#include "batch.hpp"

namespace qrmoe {

namespace {

constexpr int kShrinkStep = 64;                // values of K a wave takes at a time: one cache line of a row
constexpr int kShrinkWaves = 8;
constexpr int kExpandCols = 256;

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

// Token of entry i of perm, or -1.
__device__ __forceinline__ int token_at(const LoraArgs& a, int i) {
    const int t = a.perm[i];
    return t >= 0 && t < a.T ? t : -1;
}

// RF: fragments of 16 ranks.
template <int RF>
__global__ __launch_bounds__(kShrinkWaves* kWave) void lora_shrink_kernel(LoraArgs a) {
    __shared__ __align__(16) float part[kShrinkWaves][RF * 256];
    const int sub = blockIdx.x % 4, split = blockIdx.y;
    Run run = load_run(a, blockIdx.x / 4);
    run.r0 += 16 * sub;
    if (run.g < 0 || run.g == a.L || run.r0 >= run.r1) return;
    const int rows = min(16, run.r1 - run.r0), j0 = blockIdx.z * (16 * RF);
    const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int S = ceil_div(a.K, kShrinkStep), slice = split * kShrinkWaves + wave, slices = a.splits * kShrinkWaves;
    const int s_beg = static_cast<long long>(S) * slice / slices, s_end = static_cast<long long>(S) * (slice + 1) / slices;

    const uint16_t* arow[RF];
#pragma unroll
    for (int f = 0; f < RF; ++f)
        arow[f] = a.a + (static_cast<size_t>(run.g) * a.r + min(j0 + 16 * f + col, a.r - 1)) * a.K;
    const int t = max(token_at(a, run.r0 + min(col, rows - 1)), 0);
    const uint16_t* xrow = a.x + t * a.x_stride;
    f32x4 acc[RF];
#pragma unroll
    for (int f = 0; f < RF; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
    // 16 bytes of a row from value k on, zeros past K (a multiple of 32)
    auto chunk = [&](const uint16_t* row, int k) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(row + (k < a.K ? k : 0));
        return bf16x8_from_u32x4(k < a.K ? v : u32x4{0u, 0u, 0u, 0u});
    };
#pragma unroll 2
    for (int s = s_beg; s < s_end; ++s) {
        const int k = s * kShrinkStep + 8 * g;
        const bf16x8 x0 = chunk(xrow, k), x1 = chunk(xrow, k + 32);
#pragma unroll
        for (int f = 0; f < RF; ++f) {
            acc[f] = mfma16x16x32(chunk(arow[f], k), x0, acc[f]);
            acc[f] = mfma16x16x32(chunk(arow[f], k + 32), x1, acc[f]);
        }
    }
    // value [token col][rank 16 f + 4 g + i]
#pragma unroll
    for (int f = 0; f < RF; ++f) *reinterpret_cast<f32x4*>(&part[wave][col * 16 * RF + 16 * f + 4 * g]) = acc[f];
    __syncthreads();
    for (int i = threadIdx.x; i < rows * 16 * RF; i += kShrinkWaves * kWave) {
        const int j = j0 + i % (16 * RF);
        if (j >= a.r) continue;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kShrinkWaves; ++w) v += part[w][i];
        a.v[(static_cast<size_t>(split) * a.T + run.r0 + i / (16 * RF)) * a.r + j] = v;
    }
}

// Three bf16 parts of eight floats, exact to 2^-24: each subtraction is exact
// and each part takes the next 8 bits.
__device__ __forceinline__ void split_parts(const f32x4& lo, const f32x4& hi, bf16x8 (&p)[3]) {
    u32x4 w[3];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f32x2 v = i < 2 ? f32x2{lo[2 * i], lo[2 * i + 1]} : f32x2{hi[2 * i - 4], hi[2 * i - 3]};
#pragma unroll
        for (int q = 0; q < 3; ++q) {
            w[q][i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
            v = f32x2{v[0] - bf16lo(w[q][i]), v[1] - bf16hi(w[q][i])};
        }
    }
#pragma unroll
    for (int q = 0; q < 3; ++q) p[q] = bf16x8_from_u32x4(w[q]);
}

// Eight neighbouring values of base or out.
template <bool F32>
struct Eight {
    f32x4 lo, hi;
    __device__ __forceinline__ void load(const void* base, long long at, int n, bool vec) {
        if constexpr (F32) {
            const float* p = static_cast<const float*>(base) + at;
            if (vec && n >= 8) {
                lo = *reinterpret_cast<const f32x4*>(p);
                hi = *reinterpret_cast<const f32x4*>(p + 4);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    lo[i] = i < n ? p[i] : 0.f;
                    hi[i] = 4 + i < n ? p[4 + i] : 0.f;
                }
            }
        } else {
            const uint16_t* p = static_cast<const uint16_t*>(base) + at;
            u32x4 w;
            if (vec && n >= 8) {
                w = *reinterpret_cast<const u32x4*>(p);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = (2 * i < n ? p[2 * i] : 0u) | (2 * i + 1 < n ? static_cast<uint32_t>(p[2 * i + 1]) << 16 : 0u);
            }
            lo = f32x4{bf16lo(w[0]), bf16hi(w[0]), bf16lo(w[1]), bf16hi(w[1])};
            hi = f32x4{bf16lo(w[2]), bf16hi(w[2]), bf16lo(w[3]), bf16hi(w[3])};
        }
    }
    __device__ __forceinline__ void store(void* out, long long at, int n, bool vec) const {
        if constexpr (F32) {
            float* p = static_cast<float*>(out) + at;
            if (vec && n >= 8) {
                *reinterpret_cast<f32x4*>(p) = lo;
                *reinterpret_cast<f32x4*>(p + 4) = hi;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i < n) p[i] = lo[i];
                    if (4 + i < n) p[4 + i] = hi[i];
                }
            }
        } else {
            uint16_t* p = static_cast<uint16_t*>(out) + at;
            const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            if (vec && n >= 8) {
                u32x4 w;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = f32_to_bf16_rne(v[2 * i]) | static_cast<uint32_t>(f32_to_bf16_rne(v[2 * i + 1])) << 16;
                *reinterpret_cast<u32x4*>(p) = w;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < n) p[i] = f32_to_bf16_rne(v[i]);
            }
        }
    }
};

// A wave's 64 columns from n0 on and 16 TT tokens.  Fragment f of 16 weight rows
// holds columns 32 (f/2) + 8 (row/4) + 4 (f%2) + row%4, so the two fragments of a
// pair give a lane eight neighbouring columns of its token.
template <bool F32, int TT>
__device__ __forceinline__ void expand_body(const LoraArgs& a, const Run& run, int n0) {
    const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
    const uint16_t* brow[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
        const int n = n0 + 32 * (f / 2) + 8 * (col / 4) + 4 * (f % 2) + col % 4;
        brow[f] = a.b + (static_cast<size_t>(run.g) * a.N + min(n, a.N - 1)) * a.r;
    }
    int t[TT];
    Eight<F32> base[TT][2];
#pragma unroll
    for (int q = 0; q < TT; ++q) {
        const int i = run.r0 + 16 * q + col;
        t[q] = i < run.r1 ? token_at(a, i) : -1;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int n = n0 + 32 * p + 8 * g;
            if (t[q] >= 0 && n < a.N) base[q][p].load(a.base, t[q] * a.base_stride + n, a.N - n, a.vec);
        }
    }
    f32x4 acc[4][TT];
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
        for (int q = 0; q < TT; ++q) acc[f][q] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int j = 8 * g; j - 8 * g < a.r; j += 32) {
        const bool live = j < a.r;             // r is a multiple of 8
        bf16x8 w[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(brow[f] + (live ? j : 0));
            w[f] = bf16x8_from_u32x4(live ? v : u32x4{0u, 0u, 0u, 0u});
        }
#pragma unroll
        for (int q = 0; q < TT; ++q) {
            f32x4 lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
            if (live) {
                const float* v = a.v + static_cast<size_t>(min(run.r0 + 16 * q + col, run.r1 - 1)) * a.r + j;
                for (int s = 0; s < a.splits; ++s) {
                    const f32x4* p = reinterpret_cast<const f32x4*>(v + static_cast<size_t>(s) * a.T * a.r);
                    lo += p[0];
                    hi += p[1];
                }
            }
            bf16x8 parts[3];
            split_parts(lo, hi, parts);
#pragma unroll
            for (int f = 0; f < 4; ++f)
#pragma unroll
                for (int p = 2; p >= 0; --p) acc[f][q] = mfma16x16x32(w[f], parts[p], acc[f][q]);
        }
    }
    const float scale = a.scales ? a.scales[run.g] : 1.f;
#pragma unroll
    for (int q = 0; q < TT; ++q) {
        if (t[q] < 0) continue;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int n = n0 + 32 * p + 8 * g;
            if (n >= a.N) continue;
            Eight<F32> o = base[q][p];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                o.lo[i] = fmaf(scale, acc[2 * p][q][i], o.lo[i]);
                o.hi[i] = fmaf(scale, acc[2 * p + 1][q][i], o.hi[i]);
            }
            o.store(a.out, t[q] * a.out_stride + n, a.N - n, a.vec);
        }
    }
}

// Rows of no adapter: base as it is, 64 columns of a wave.
template <bool F32>
__device__ __forceinline__ void copy_body(const LoraArgs& a, const Run& run, int n0) {
    const int lane = threadIdx.x & 63, n = n0 + 8 * (lane & 7);
    if (n >= a.N) return;
    for (int i = run.r0 + (lane >> 3); i < run.r1; i += 8) {
        const int t = token_at(a, i);
        if (t < 0) continue;
        Eight<F32> v;
        v.load(a.base, t * a.base_stride + n, a.N - n, a.vec);
        v.store(a.out, t * a.out_stride + n, a.N - n, a.vec);
    }
}

template <bool F32>
__global__ __launch_bounds__(256) void lora_expand_kernel(LoraArgs a, int n_tiles) {
    const Run run = load_run(a, blockIdx.x / n_tiles);
    if (run.g < 0) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x % n_tiles * kExpandCols + 64 * wave;
    if (n0 >= a.N) return;
    if (run.g == a.L) {
        if (!a.in_place) copy_body<F32>(a, run, n0);
        return;
    }
    const int rows = run.r1 - run.r0;
    if (rows > 32) expand_body<F32, 4>(a, run, n0);
    else if (rows > 16) expand_body<F32, 2>(a, run, n0);
    else expand_body<F32, 1>(a, run, n0);
}

template <int RF>
void launch_shrink(const LoraArgs& a, hipStream_t st) {
    const dim3 grid(a.n_items * 4, a.splits, ceil_div(a.r, 16 * RF));
    lora_shrink_kernel<RF><<<grid, kShrinkWaves * kWave, 0, st>>>(a);
}

}  // namespace

int lora_splits(int T, int K, int r, int L) {
    const int groups = L < T ? L : T, steps = ceil_div(K, kShrinkStep);
    const int runs = ceil_div(T, 16) + groups / 2;         // taking it that half of the adapters end in a partial run
    int s = 1;
    while (s < 8 && runs * s * 2 <= 512 && steps >= kShrinkWaves * s * 2) s *= 2;
    return s;
}

hipError_t launch_lora_add(const LoraArgs& a, hipStream_t st) {
    if (a.r <= 16) launch_shrink<1>(a, st);
    else if (a.r <= 32) launch_shrink<2>(a, st);
    else launch_shrink<4>(a, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int n_tiles = ceil_div(a.N, kExpandCols), blocks = a.n_items * n_tiles;
    if (a.f32) lora_expand_kernel<true><<<blocks, 256, 0, st>>>(a, n_tiles);
    else lora_expand_kernel<false><<<blocks, 256, 0, st>>>(a, n_tiles);
    return hipGetLastError();
}

}  // namespace qrmoe
