// Entry points of the FP8 operators: argument checks (all on the host, before
// any HIP call) and launches.  See include/moe_fp8.h for the contract.
#include <cmath>

#include "../../include/moe_fp8.h"
#include "fp8.hpp"
#include "kernels.hpp"
#include "validate.hpp"
#include "workspace.hpp"

namespace qrmoe {
namespace {

using check::aligned;

int hip_rc(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

bool known_type(int t) { return t == MOE_TYPE_BF16 || t == MOE_TYPE_F32; }

constexpr int kDimLimit = 1 << 30;
constexpr int kDepthLimit = 1 << 22;      // 256 weight rows within a 32-bit offset

// Sizes of one product: N weight rows of depth K.
int check_dims(int N, int K) {
    if (N < 1 || N >= kDimLimit || K < 32 || K % 32 || K > kDepthLimit) return MOE_ERR_SHAPE;
    return MOE_OK;
}

int check_operands(const uint8_t* a, const float* a_scales, const uint8_t* w, const float* w_scales) {
    if (!a || !a_scales || !w || !w_scales) return MOE_ERR_NULL;
    if (!aligned(a, 16) || !aligned(w, 16) || !aligned(a_scales, 4) || !aligned(w_scales, 4)) return MOE_ERR_ALIGN;
    return MOE_OK;
}

int run_product(const Fp8Args& a, bool gate_up, hipStream_t st) {
    const Fp8Plan p = fp8_plan(a, gate_up);
    if (p.blocks >= kMostBlocks) return MOE_ERR_SHAPE;
    return hip_rc(p.path == Fp8Path::kFew ? launch_fp8_few(a, p, gate_up, st) : launch_fp8_tile(a, p, gate_up, st));
}

Fp8Args grouped_args(int R, int E, int N, int K, const uint8_t* a, int a_rows, const float* a_scales, const uint8_t* w,
                     const float* w_scales, const int32_t* offsets, const int32_t* perm, int k) {
    Fp8Args p{};
    p.R = R;
    p.E = E;
    p.N = N;
    p.K = K;
    p.a = a;
    p.a_stride = K;
    p.a_rows = a_rows;
    p.a_scales = a_scales;
    p.w[0] = w;
    p.w_scales[0] = w_scales;
    p.offsets = offsets;
    p.perm = perm;
    p.k = k;
    return p;
}

void set_out(Fp8Args& p, void* out, int out_type, long long out_stride) {
    p.out = out;
    p.out_stride = out_stride;
    p.out_f32 = out_type == MOE_TYPE_F32;
    p.out_vec = out_stride % 4 == 0;
}

Fp8Args gate_up_args(const moe_shape& s, const uint8_t* a, const float* a_scales, const uint8_t* gate,
                     const float* gate_scales, const uint8_t* up, const float* up_scales, const int32_t* offsets,
                     const int32_t* perm, uint8_t* act, float* act_scales, void* ws) {
    Fp8Args p = grouped_args(s.T * s.k, s.E, s.f, s.d, a, s.T, a_scales, gate, gate_scales, offsets, perm, s.k);
    p.w[1] = up;
    p.w_scales[1] = up_scales;
    p.act = act;
    p.act_scales = act_scales;
    if (fp8_plan(p, true).path != Fp8Path::kMany) {
        p.hidden = static_cast<float*>(ws);
        p.flags = reinterpret_cast<unsigned long long*>(static_cast<char*>(ws) + fp8_hidden_bytes(p));
    }
    return p;
}

// Workspace of a gate/up call: none where a workgroup has whole runs.
size_t hidden_bytes(const moe_shape& s) {
    static const int32_t grouped = 0;      // stands for offsets: only its presence counts
    Fp8Args p{};
    p.R = s.T * s.k;
    p.E = s.E;
    p.N = s.f;
    p.K = s.d;
    p.offsets = &grouped;
    return p.R && fp8_plan(p, true).path != Fp8Path::kMany ? fp8_hidden_bytes(p) + fp8_flag_bytes(p) : 0;
}

struct Fp8LayerCarve {
    size_t offsets, perm, inv, act, act_scales, hidden, y, total;
};

Fp8LayerCarve fp8_layer_carve(const moe_shape& s) {
    Fp8LayerCarve c;
    const size_t R = static_cast<size_t>(s.T) * s.k;
    c.offsets = kHeader;
    c.perm = c.offsets + align256(static_cast<size_t>(s.E + 1) * 4);
    c.inv = c.perm + align256(R * 4);
    c.act = c.inv + align256(R * 4);
    c.act_scales = c.act + align256(R * s.f);
    c.hidden = c.act_scales + align256(R * ceil_div(s.f, kRun) * 4);
    c.y = c.hidden + hidden_bytes(s);
    c.total = c.y + align256(R * s.d * 4);
    return c;
}

int check_gate_up(const moe_shape& s, const uint8_t* a, const float* a_scales, const uint8_t* gate,
                  const float* gate_scales, const uint8_t* up, const float* up_scales, const int32_t* offsets,
                  const int32_t* perm, const uint8_t* act, const float* act_scales, const void* ws, size_t ws_bytes) {
    int rc;
    if ((rc = check_dims(s.f, s.d)) != MOE_OK) return rc;
    if ((rc = check_operands(a, a_scales, gate, gate_scales)) != MOE_OK) return rc;
    if ((rc = check_operands(a, a_scales, up, up_scales)) != MOE_OK) return rc;
    if (!offsets || !perm || !act || !act_scales) return MOE_ERR_NULL;
    if (!aligned(offsets, 4) || !aligned(perm, 4) || !aligned(act, 16) || !aligned(act_scales, 4)) return MOE_ERR_ALIGN;
    const size_t need = hidden_bytes(s);
    if (need) {
        if (!ws) return MOE_ERR_NULL;
        if (!aligned(ws, 16)) return MOE_ERR_ALIGN;
        if (ws_bytes < need) return MOE_ERR_WORKSPACE;
    }
    return MOE_OK;
}

// Rows of `stride` values (of `bytes` each): whole 16-byte units apart.
bool stride_ok(int64_t stride, int bytes, int64_t least) { return stride >= least && stride * bytes % 16 == 0; }

}  // namespace
}  // namespace qrmoe

using namespace qrmoe;

extern "C" {

int moe_add_rmsnorm(int32_t T, int32_t d, const void* x, int32_t x_type, int64_t x_stride, const void* residual,
                    void* residual_out, int32_t residual_type, int64_t residual_stride, int64_t residual_out_stride,
                    const void* weight, int32_t weight_type, float eps, uint16_t* y, uint8_t* q, float* q_scales,
                    hipStream_t stream) {
    if (T < 0 || d < 32 || d % 32 || d > (1 << 20) || !std::isfinite(eps) || eps < 0.f) return MOE_ERR_SHAPE;
    if (T == 0) return MOE_OK;
    if (!x || !residual != !residual_out || !q != !q_scales || (!y && !q && !residual_out)) return MOE_ERR_NULL;
    if (!known_type(x_type) || (residual && !known_type(residual_type)) || (weight && !known_type(weight_type)))
        return MOE_ERR_FORMAT;
    const int xb = x_type == MOE_TYPE_F32 ? 4 : 2, rb = residual_type == MOE_TYPE_F32 ? 4 : 2;
    const int64_t most = int64_t{1} << 40;
    if (!stride_ok(x_stride, xb, 0) || x_stride > most || (x_stride && x_stride < d)) return MOE_ERR_SHAPE;
    if (residual) {
        if (!stride_ok(residual_stride, rb, 0) || residual_stride > most || (residual_stride && residual_stride < d))
            return MOE_ERR_SHAPE;
        if (!stride_ok(residual_out_stride, rb, d) || residual_out_stride > most) return MOE_ERR_SHAPE;
        if (residual == residual_out && residual_stride != residual_out_stride) return MOE_ERR_UNSUPPORTED;
    }
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(residual_out, 16) || !aligned(weight, 16) ||
        !aligned(y, 16) || !aligned(q, 16) || !aligned(q_scales, 4))
        return MOE_ERR_ALIGN;
    NormArgs a{T, d, x, residual, weight, residual_out, x_stride, residual_stride, residual_out_stride, eps, y, q, q_scales};
    return hip_rc(launch_add_rmsnorm(a, x_type == MOE_TYPE_F32, residual && residual_type == MOE_TYPE_F32,
                                     weight && weight_type == MOE_TYPE_F32, stream));
}

int moe_gemm_fp8(int32_t M, int32_t N, int32_t K, const uint8_t* a, int64_t a_stride, const float* a_scales,
                 const uint8_t* w, const float* w_scales, void* out, int32_t out_type, int64_t out_stride,
                 hipStream_t stream) {
    int rc;
    if (M < 0 || M >= kDimLimit) return MOE_ERR_SHAPE;
    if ((rc = check_dims(N, K)) != MOE_OK) return rc;
    if (M == 0) return MOE_OK;
    if ((rc = check_operands(a, a_scales, w, w_scales)) != MOE_OK) return rc;
    if (!out) return MOE_ERR_NULL;
    if (!known_type(out_type)) return MOE_ERR_FORMAT;
    const int64_t most = int64_t{1} << 40;
    if (!stride_ok(a_stride, 1, K) || a_stride > most || out_stride < N || out_stride > most) return MOE_ERR_SHAPE;
    if (!aligned(out, 16)) return MOE_ERR_ALIGN;
    Fp8Args p = grouped_args(M, 1, N, K, a, M, a_scales, w, w_scales, nullptr, nullptr, 1);
    p.a_stride = a_stride;
    set_out(p, out, out_type, out_stride);
    return run_product(p, false, stream);
}

int moe_grouped_gemm_fp8(int32_t R, int32_t E, int32_t N, int32_t K, const uint8_t* a, int32_t a_rows,
                         const float* a_scales, const uint8_t* w, const float* w_scales, const int32_t* offsets,
                         const int32_t* perm, int32_t k, void* out, int32_t out_type, hipStream_t stream) {
    int rc;
    if (R < 0 || R >= kDimLimit || E < 1 || E > kMaxExperts || k < 1 || a_rows < 1 || (!perm && a_rows < R))
        return MOE_ERR_SHAPE;
    if ((rc = check_dims(N, K)) != MOE_OK) return rc;
    if (R == 0) return MOE_OK;
    if ((rc = check_operands(a, a_scales, w, w_scales)) != MOE_OK) return rc;
    if (!offsets || !out) return MOE_ERR_NULL;
    if (!known_type(out_type)) return MOE_ERR_FORMAT;
    if (!aligned(offsets, 4) || !aligned(perm, 4) || !aligned(out, 16)) return MOE_ERR_ALIGN;
    Fp8Args p = grouped_args(R, E, N, K, a, a_rows, a_scales, w, w_scales, offsets, perm, k);
    set_out(p, out, out_type, N);
    return run_product(p, false, stream);
}

size_t moe_expert_gate_up_fp8_workspace_bytes(const moe_shape* shape) {
    return check::check_shape(shape) == MOE_OK ? hidden_bytes(*shape) : 0;
}

int moe_expert_gate_up_fp8(const moe_shape* shape, const uint8_t* a, const float* a_scales, const uint8_t* gate,
                           const float* gate_scales, const uint8_t* up, const float* up_scales,
                           const int32_t* offsets, const int32_t* perm, uint8_t* act, float* act_scales, void* ws,
                           size_t ws_bytes, hipStream_t stream) {
    int rc = check::check_shape(shape);
    if (rc != MOE_OK) return rc;
    if (shape->T == 0) return MOE_OK;
    if ((rc = check_gate_up(*shape, a, a_scales, gate, gate_scales, up, up_scales, offsets, perm, act, act_scales, ws,
                            ws_bytes)) != MOE_OK)
        return rc;
    return run_product(gate_up_args(*shape, a, a_scales, gate, gate_scales, up, up_scales, offsets, perm, act,
                                    act_scales, ws),
                       true, stream);
}

size_t moe_layer_fp8_workspace_bytes(const moe_shape* shape) {
    return check::check_shape(shape) == MOE_OK ? fp8_layer_carve(*shape).total : 0;
}

int moe_layer_fp8(const moe_shape* shape, const uint16_t* x, const uint8_t* xq, const float* xq_scales,
                  const float* w_router, const float* bias, float* logits, const moe_fp8_experts* experts,
                  int32_t* topk_ids, float* topk_w, float* out, void* ws, size_t ws_bytes, hipStream_t stream) {
    int rc = check::check_shape(shape);
    if (rc != MOE_OK) return rc;
    if (shape->T == 0) return MOE_OK;
    const moe_shape& s = *shape;
    if (!experts || !ws || !out) return MOE_ERR_NULL;
    if (!aligned(ws, 16) || !aligned(out, 16)) return MOE_ERR_ALIGN;
    const Fp8LayerCarve c = fp8_layer_carve(s);
    if (ws_bytes < c.total) return MOE_ERR_WORKSPACE;
    char* base = static_cast<char*>(ws);
    int32_t* offsets = reinterpret_cast<int32_t*>(base + c.offsets);
    int32_t* perm = reinterpret_cast<int32_t*>(base + c.perm);
    int32_t* inv = reinterpret_cast<int32_t*>(base + c.inv);
    uint8_t* act = reinterpret_cast<uint8_t*>(base + c.act);
    float* act_scales = reinterpret_cast<float*>(base + c.act_scales);
    float* y = reinterpret_cast<float*>(base + c.y);
    const moe_fp8_experts& ex = *experts;
    if ((rc = check::check_route_args(s, x, w_router, bias, logits, topk_ids, topk_w)) != MOE_OK) return rc;
    if ((rc = check_gate_up(s, xq, xq_scales, ex.gate, ex.gate_scales, ex.up, ex.up_scales, offsets, perm, act,
                            act_scales, base + c.hidden, hidden_bytes(s))) != MOE_OK)
        return rc;
    if ((rc = check_dims(s.d, s.f)) != MOE_OK) return rc;
    if ((rc = check_operands(act, act_scales, ex.down, ex.down_scales)) != MOE_OK) return rc;

    if (small_route_supported(s)) {
        if ((rc = hip_rc(launch_small_route(s, x, w_router, bias, logits, topk_ids, topk_w, offsets, perm, inv,
                                            stream))) != MOE_OK)
            return rc;
    } else {
        if ((rc = hip_rc(launch_route(s, x, w_router, bias, logits, topk_ids, topk_w, stream))) != MOE_OK) return rc;
        if ((rc = hip_rc(launch_dispatch(s, topk_ids, offsets, perm, inv, static_cast<uint32_t*>(ws), stream))) != MOE_OK)
            return rc;
    }
    // both fit a grid: T*k*f < 2^31 and f <= 2^22, and so for d
    const Fp8Args gu = gate_up_args(s, xq, xq_scales, ex.gate, ex.gate_scales, ex.up, ex.up_scales, offsets, perm, act,
                                    act_scales, base + c.hidden);
    if ((rc = run_product(gu, true, stream)) != MOE_OK) return rc;
    Fp8Args down = grouped_args(s.T * s.k, s.E, s.d, s.f, act, s.T * s.k, act_scales, ex.down, ex.down_scales, offsets,
                                nullptr, 1);
    set_out(down, y, MOE_TYPE_F32, s.d);
    if ((rc = run_product(down, false, stream)) != MOE_OK) return rc;
    return hip_rc(launch_combine(s, y, inv, topk_w, out, stream));
}

}  // extern "C"
