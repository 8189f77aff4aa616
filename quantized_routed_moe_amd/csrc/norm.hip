// Residual addition with root-mean-square norm and an E4M3 output
// (moe_add_rmsnorm).  Per row: h = x + residual rounded to the residual's
// type and stored, v = h / sqrt(mean h^2 + eps) * w, y = bf16(v), and per run
// of 128 values the scale max|v| / 448 with the codes v / scale.
//
// Bound by HBM at many rows: each input is read and each output written once
// (T * d * 11 bytes for fp32 x, a bf16 stream and both outputs: 2048 x 4096 in
// 19 us, 4.8 TB/s; a large copy reaches 5.2).  One workgroup takes a row and
// keeps it in registers between the sum of squares and the outputs; a thread
// holds 8 consecutive values per chunk, so a run of 128 is 16 neighbouring
// lanes and its maximum four lane exchanges.  Few rows are bound by the length
// of a thread's work, mostly the divisions of its codes: the row is spread over
// as many threads as it has chunks (1 x 4096: 3.5 us, of which a launch of any
// size is 2.7; with two chunks a thread, in one run, 5.3 beside 4.1).
#include "fp8.hpp"
#include "kernels.hpp"

namespace qrmoe {

namespace {

struct F8 {
    float v[8];
};

template <bool F32>
__device__ __forceinline__ F8 load8(const void* base, long long i) {
    F8 r;
    if constexpr (F32) {
        const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(base) + i);
        const f32x4 a = p[0], b = p[1];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r.v[j] = a[j];
            r.v[4 + j] = b[j];
        }
    } else {
        const u32x4 a = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r.v[2 * j] = bf16lo(a[j]);
            r.v[2 * j + 1] = bf16hi(a[j]);
        }
    }
    return r;
}

__device__ __forceinline__ u32x4 pack_bf16(const F8& f) {
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        o[j] = f32_to_bf16_rne(f.v[2 * j]) | static_cast<uint32_t>(f32_to_bf16_rne(f.v[2 * j + 1])) << 16;
    return o;
}

// x + residual, rounded to the residual's type and stored.
template <bool XF, bool RF>
__device__ __forceinline__ F8 add_residual(const NormArgs& a, int t, int i) {
    F8 h = load8<XF>(a.x, t * a.x_stride + i);
    if (a.res) {
        const F8 r = load8<RF>(a.res, t * a.res_stride + i);
#pragma unroll
        for (int j = 0; j < 8; ++j) h.v[j] += r.v[j];
        if constexpr (RF) {
            f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(a.res_out) + t * a.res_out_stride + i);
            p[0] = f32x4{h.v[0], h.v[1], h.v[2], h.v[3]};
            p[1] = f32x4{h.v[4], h.v[5], h.v[6], h.v[7]};
        } else {
            const u32x4 w = pack_bf16(h);
            *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.res_out) + t * a.res_out_stride + i) = w;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h.v[2 * j] = bf16lo(w[j]);
                h.v[2 * j + 1] = bf16hi(w[j]);
            }
        }
    }
    return h;
}

// Outputs of the 8 values at column i (live: i < d).  All 16 lanes of a run
// take part in its maximum.
template <bool WF>
__device__ __forceinline__ void emit(const NormArgs& a, int t, int i, bool live, const F8& h, float rstd) {
    F8 v;
    if (live) {
        F8 w;
        if (a.weight) w = load8<WF>(a.weight, i);
#pragma unroll
        for (int j = 0; j < 8; ++j) v.v[j] = h.v[j] * rstd * (a.weight ? w.v[j] : 1.f);
        if (a.y) *reinterpret_cast<u32x4*>(a.y + static_cast<long long>(t) * a.d + i) = pack_bf16(v);
    }
    if (!a.q) return;
    float m = 0.f;
    if (live) {
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v.v[j]));
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
    if (!live) return;
    const float s = run_scale(m);
    u32x2 c;
    c[0] = e4m3x4_rne(v.v[0] / s, v.v[1] / s, v.v[2] / s, v.v[3] / s);
    c[1] = e4m3x4_rne(v.v[4] / s, v.v[5] / s, v.v[6] / s, v.v[7] / s);
    *reinterpret_cast<u32x2*>(a.q + static_cast<long long>(t) * a.d + i) = c;
    if (i % kRun == 0) a.q_scales[static_cast<long long>(t) * ceil_div(a.d, kRun) + i / kRun] = s;
}

template <int THREADS>
__device__ __forceinline__ float block_sum(float v) {
    __shared__ float part[THREADS / kWave];
    v = wave_sum_f32(v);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < THREADS / kWave; ++i) s += part[i];
    return s;
}

// One row per workgroup, C chunks of 8 values per thread in registers
// (d <= 8 * THREADS * C); C = 0: any d, the row's h read a second time.
template <int THREADS, int C, bool XF, bool RF, bool WF>
__global__ __launch_bounds__(THREADS) void norm_kernel(NormArgs a) {
    const int t = blockIdx.x, i0 = threadIdx.x * 8;
    constexpr int kStep = THREADS * 8;
    float ss = 0.f;
    if constexpr (C > 0) {
        F8 h[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = i0 + c * kStep;
            if (i < a.d) {
                h[c] = add_residual<XF, RF>(a, t, i);
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(h[c].v[j], h[c].v[j], ss);
            }
        }
        const float rstd = 1.f / sqrtf(block_sum<THREADS>(ss) / a.d + a.eps);
#pragma unroll
        for (int c = 0; c < C; ++c) emit<WF>(a, t, i0 + c * kStep, i0 + c * kStep < a.d, h[c], rstd);
    } else {
        for (int i = i0; i < a.d; i += kStep) {
            const F8 h = add_residual<XF, RF>(a, t, i);
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(h.v[j], h.v[j], ss);
        }
        const float rstd = 1.f / sqrtf(block_sum<THREADS>(ss) / a.d + a.eps);
        for (int base = 0; base < a.d; base += kStep) {
            const int i = base + i0;
            F8 h;
            if (i < a.d) {
                // the thread's own store of the first pass, or x itself
                h = a.res ? load8<RF>(a.res_out, t * a.res_out_stride + i) : load8<XF>(a.x, t * a.x_stride + i);
            }
            emit<WF>(a, t, i, i < a.d, h, rstd);
        }
    }
}

// A grid holds fewer than 2^32 threads: rows beyond that go into further
// launches, all of the kernel that the whole call's size chooses.
template <int THREADS, int C, bool XF, bool RF, bool WF>
hipError_t launch_rows(const NormArgs& a, hipStream_t st) {
    constexpr long long kMost = (1ll << 31) / THREADS;
    const long long xb = XF ? 4 : 2, rb = RF ? 4 : 2;
    for (long long t = 0; t < a.T; t += kMost) {
        NormArgs b = a;
        b.T = static_cast<int>(a.T - t < kMost ? a.T - t : kMost);
        b.x = static_cast<const char*>(a.x) + t * a.x_stride * xb;
        if (a.res) {
            b.res = static_cast<const char*>(a.res) + t * a.res_stride * rb;
            b.res_out = static_cast<char*>(a.res_out) + t * a.res_out_stride * rb;
        }
        if (a.y) b.y = a.y + t * a.d;
        if (a.q) {
            b.q = a.q + t * a.d;
            b.q_scales = a.q_scales + t * ceil_div(a.d, kRun);
        }
        norm_kernel<THREADS, C, XF, RF, WF><<<b.T, THREADS, 0, st>>>(b);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <bool XF, bool RF, bool WF>
hipError_t launch(const NormArgs& a, hipStream_t st) {
    // One chunk a thread up to 4096 (2048 rows: 19.4 us, two 20.3), and up to
    // 8192 while there is no more than one row a CU (64 rows: one 5.7, two
    // 6.3; 2048 rows: 39.6, 36.9).  Longer rows are read again: chunks held in
    // registers took as long (1 x 20000: 9.0, 8.9) or longer (1024 rows: 54,
    // 50), and 256 threads 17.5 and 59.
    if (a.d <= 2048) return launch_rows<256, 1, XF, RF, WF>(a, st);
    if (a.d <= 4096) return launch_rows<512, 1, XF, RF, WF>(a, st);
    if (a.d <= 8192 && a.T <= 256) return launch_rows<1024, 1, XF, RF, WF>(a, st);
    if (a.d <= 8192) return launch_rows<512, 2, XF, RF, WF>(a, st);
    return launch_rows<1024, 0, XF, RF, WF>(a, st);
}

template <bool XF, bool RF>
hipError_t launch_w(const NormArgs& a, bool w_f32, hipStream_t st) {
    return w_f32 ? launch<XF, RF, true>(a, st) : launch<XF, RF, false>(a, st);
}

}  // namespace

hipError_t launch_add_rmsnorm(const NormArgs& a, bool x_f32, bool res_f32, bool w_f32, hipStream_t st) {
    if (x_f32) return res_f32 ? launch_w<true, true>(a, w_f32, st) : launch_w<true, false>(a, w_f32, st);
    return res_f32 ? launch_w<false, true>(a, w_f32, st) : launch_w<false, false>(a, w_f32, st);
}

}  // namespace qrmoe
