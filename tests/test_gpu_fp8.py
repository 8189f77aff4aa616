"""The FP8 operators on the GPU against float64 (tests/fp8_ref.py), at the
sizes, strides and routings where a tile, a run or a group can go wrong."""

import ctypes

import pytest
import torch

import fp8_ref as R8
import quantized_routed_moe_amd as qm
from fp8_ref import gen, runs

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------- norm

def norm_case(T, d, xt, rt, wt, seed=0, scale=3.0):
    g = gen(seed)
    x = (scale * torch.randn((T, d), generator=g, device="cuda")).to(xt)
    res = None if rt is None else (scale * torch.randn((T, d), generator=g, device="cuda")).to(rt)
    w = None if wt is None else (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(wt)
    return x, res, w


def check_norm(x, res, w, eps, got):
    y, h, q, sc = got
    want_h, v, dv = R8.norm(x, res, w, eps)
    if res is not None:
        assert torch.equal(h, want_h)
    R8.check_rounded(y, v, dv, BF16, "y")
    if q is not None:
        R8.check_quantised(q, sc, v, dv, "q")


@pytest.mark.parametrize("T,d", [(1, 32), (3, 96), (5, 128), (7, 160), (2, 2048), (4, 2080), (333, 1056), (9, 4096),
                                 (2, 4128), (3, 8192), (2, 8224), (1, 20000), (2, 65536), (2048, 256)])
@pytest.mark.parametrize("xt,rt,wt", [(F32, BF16, BF16), (BF16, F32, F32), (BF16, None, None), (F32, F32, None),
                                      (BF16, BF16, F32), (F32, None, BF16)])
def test_norm(T, d, xt, rt, wt):
    x, res, w = norm_case(T, d, xt, rt, wt, seed=d + T)
    check_norm(x, res, w, 1e-6, qm.add_rmsnorm(x, w, residual=res, eps=1e-6, fp8=True))


@pytest.mark.parametrize("T,d", [(256, 8192), (257, 4128), (300, 8192), (70, 8224)])
def test_norm_of_many_long_rows(T, d):
    x, res, w = norm_case(T, d, F32, BF16, BF16, seed=d + T)
    check_norm(x, res, w, 1e-6, qm.add_rmsnorm(x, w, residual=res, eps=1e-6, fp8=True))


def test_norm_outputs_alone():
    x, res, w = norm_case(6, 416, F32, BF16, BF16)
    y, h, q, sc = qm.add_rmsnorm(x, w, residual=res, fp8=True)
    only_y = qm.add_rmsnorm(x, w, residual=res)
    assert torch.equal(only_y[0], y) and only_y[2] is None and only_y[3] is None
    only_q = qm.add_rmsnorm(x, w, residual=res, y=False, fp8=True)
    assert only_q[0] is None and torch.equal(only_q[2].view(torch.uint8), q.view(torch.uint8)) and torch.equal(only_q[3], sc)
    only_h = qm.add_rmsnorm(x, w, residual=res, y=False)
    assert torch.equal(only_h[1], h) and only_h[0] is None


@pytest.mark.parametrize("rt", [BF16, F32])
@pytest.mark.parametrize("d", [512, 9216])
def test_norm_in_place_and_strided(rt, d):
    T = 5
    x, res, w = norm_case(T, d, BF16, rt, BF16)
    want = qm.add_rmsnorm(x, w, residual=res, fp8=True)
    # rows apart, in buffers whose other columns stay as they were
    bx = torch.zeros((T, d + 64), dtype=BF16, device="cuda")
    br = torch.full((T, d + 32), 7.0, dtype=rt, device="cuda")
    bx[:, 16:16 + d] = x
    br[:, :d] = res
    got = qm.add_rmsnorm(bx[:, 16:16 + d], w, residual=br[:, :d], residual_out=br[:, :d], fp8=True)
    for a, b in zip(want, got):
        assert torch.equal(a.view(torch.uint8) if a.dtype == torch.float8_e4m3fn else a,
                           b.view(torch.uint8) if b.dtype == torch.float8_e4m3fn else b)
    assert (br[:, d:] == 7).all() and torch.equal(br[:, :d], want[1])
    # one row of x for all
    one = qm.add_rmsnorm(x[:1].expand(T, d), w, residual=res)
    assert torch.equal(one[1], (x[:1].float() + res.float()).to(rt))


def test_norm_of_zeros_tiny_and_non_finite_rows():
    d = 384
    x = torch.zeros((5, d), dtype=F32, device="cuda")
    x[1] = 1e-30                      # far below eps: v about 1e-27, scale and codes still exact
    x[2] = 1.0
    x[2, 130] = float("nan")
    x[3] = 2.0
    x[3, 5] = float("inf")
    x[4] = 3.0
    y, _, q, sc = qm.add_rmsnorm(x, eps=1e-6, fp8=True)
    assert (y[0] == 0).all() and (q[0].float() == 0).all() and (sc[0] == 2.0 ** -126).all()
    check_norm(x[1:2], None, None, 1e-6, (y[1:2], None, q[1:2], sc[1:2]))
    assert torch.isnan(y[2]).all() and torch.isnan(q[2].float()).all()       # the row's mean is NaN
    assert torch.isnan(y[3, 5]) and (y[3, 6:] == 0).all()                    # inf * 0, and x / inf
    assert torch.isnan(q[3, 5].float()) and (q[3, 6:].float() == 0).all()
    check_norm(x[4:5], None, None, 1e-6, (y[4:5], None, q[4:5], sc[4:5]))


# ------------------------------------------------------------ dense product

def gemm_case(M, N, K, seed=0):
    g = gen(seed + 7 * M + 3 * N + K)
    return (R8.codes(g, M, K), R8.scales(g, M, runs(K)), R8.codes(g, N, K), R8.scales(g, runs(N), runs(K)))


MS = [1, 2, 15, 16, 17, 32, 33, 64, 65, 129, 257, 300, 513, 5000]


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("N,K", [(1, 32), (15, 96), (16, 128), (128, 160), (130, 1056), (257, 416), (512, 2048), (1111, 256)])
@pytest.mark.parametrize("M", MS)
def test_gemm(M, N, K, out_dtype):
    a, a_s, w, w_s = gemm_case(M, N, K)
    want, bound = R8.product(a, a_s, w, w_s, fast=out_dtype == BF16)
    R8.check_rounded(qm.gemm_fp8(a, a_s, w, w_s, out_dtype=out_dtype), want, bound, out_dtype, f"{M}x{N}x{K}")


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("M", [1, 5, 40, 700, 2048])
def test_gemm_long(M, out_dtype):
    a, a_s, w, w_s = gemm_case(M, 4096, 4096)
    want, bound = R8.product(a, a_s, w, w_s, fast=out_dtype == BF16)
    got = qm.gemm_fp8(a, a_s, w, w_s, out_dtype=out_dtype)
    R8.check_rounded(got, want, bound, out_dtype)
    assert torch.equal(got, qm.gemm_fp8(a.view(torch.uint8), a_s, w.view(torch.uint8), w_s, out_dtype=out_dtype))


@pytest.mark.parametrize("M", [3, 70, 400])
@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("pad", [1, 4, 13])
def test_gemm_strided_rows(M, out_dtype, pad):
    N, K = 300, 288
    a, a_s, w, w_s = gemm_case(M, N, K)
    big_a = torch.full((M, K + 48), 0x7F, dtype=torch.uint8, device="cuda")      # NaN codes between the rows
    big_a[:, :K] = a.view(torch.uint8)
    big = torch.full((M + 2, N + pad), 5.0, dtype=out_dtype, device="cuda")
    qm.gemm_fp8(big_a[:, :K], a_s, w, w_s, out=big[:M, :N])
    assert torch.equal(big[:M, :N], qm.gemm_fp8(a, a_s, w, w_s, out_dtype=out_dtype))
    assert (big[M:] == 5).all() and (big[:, N:] == 5).all()


@pytest.mark.parametrize("M", [4, 100, 600])
@pytest.mark.parametrize("out_dtype", [BF16, F32])
def test_gemm_nan_and_zero_scales(M, out_dtype):
    N, K = 272, 320
    a, a_s, w, w_s = gemm_case(M, N, K)
    clean = qm.gemm_fp8(a, a_s, w, w_s, out_dtype=out_dtype)
    ua, uw = a.view(torch.uint8).clone(), w.view(torch.uint8).clone()
    ua[1, 319] = 0x7F
    uw[200, 0] = 0xFF
    got = qm.gemm_fp8(ua, a_s, uw, w_s, out_dtype=out_dtype)
    hit = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    hit[1] = True
    hit[:, 200] = True
    assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], clean[~hit])
    assert (qm.gemm_fp8(a, torch.zeros_like(a_s), w, w_s, out_dtype=out_dtype) == 0).all()


def test_gemm_wide_values():
    """Codes over E4M3's whole range, where the fp8 instruction's alignment shows."""
    g = gen(3)
    M, N, K = 600, 256, 512
    mk = lambda r: (torch.randn((r, K), generator=g, device="cuda")  # noqa: E731
                    * torch.exp2(torch.randint(-9, 9, (r, K), generator=g, device="cuda").float())).clamp(-448, 448).to(torch.float8_e4m3fn)
    a, w = mk(M), mk(N)
    a_s, w_s = R8.scales(g, M, 4), R8.scales(g, 2, 4)
    for dt in (BF16, F32):
        want, bound = R8.product(a, a_s, w, w_s, fast=dt == BF16)
        R8.check_rounded(qm.gemm_fp8(a, a_s, w, w_s, out_dtype=dt), want, bound, dt)


# --------------------------------------------------------- grouped products

def grouped_ref(a, a_s, w, w_s, off, src, fast):
    off = off.tolist()
    want = torch.zeros((len(src), w.shape[1]), dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(want)
    for e in range(w.shape[0]):
        r = slice(off[e], off[e + 1])
        if off[e + 1] > off[e]:
            want[r], bound[r] = R8.product(a[src[r]], a_s[src[r]], w[e], w_s[e], fast)
    return want, bound


ROUTES = [  # T, E, k, only
    (1, 8, 2, None), (5, 64, 2, None), (3, 4, 4, None), (40, 1, 1, None), (64, 64, 6, None), (70, 3, 1, None),
    (200, 8, 2, [1, 6]), (300, 16, 1, [15]), (150, 5, 2, None), (1000, 8, 2, None), (7, 64, 1, [63])]


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("N,K", [(96, 64), (300, 416)])
@pytest.mark.parametrize("T,E,k,only", ROUTES)
def test_grouped_gemm(T, E, k, only, N, K, out_dtype):
    g = gen(T + E + k + N)
    off, perm, _ = R8.routing(g, T, E, k, only=only)
    w, w_s = R8.codes(g, E, N, K), R8.scales(g, E, runs(N), runs(K))
    fast = out_dtype == BF16
    # rows as they are
    a, a_s = R8.codes(g, T * k, K), R8.scales(g, T * k, runs(K))
    want, bound = grouped_ref(a, a_s, w, w_s, off, torch.arange(T * k, device="cuda"), fast)
    R8.check_rounded(qm.grouped_gemm_fp8(a, a_s, w, w_s, off, out_dtype=out_dtype), want, bound, out_dtype, "rows")
    # gathered from the tokens
    want, bound = grouped_ref(a[:T], a_s[:T], w, w_s, off, perm.long() // k, fast)
    got = qm.grouped_gemm_fp8(a[:T], a_s[:T].contiguous(), w, w_s, off, perm=perm, k=k, out_dtype=out_dtype)
    R8.check_rounded(got, want, bound, out_dtype, "gathered")


@pytest.mark.parametrize("R,last", [(12, 7), (600, 130), (600, 0)])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
def test_grouped_rows_past_the_last_expert_are_zero(R, last, out_dtype):
    E, N, K = 3, 272, 160
    g = gen(R)
    a, a_s, w, w_s = R8.codes(g, R, K), R8.scales(g, R, 2), R8.codes(g, E, N, K), R8.scales(g, E, 3, 2)
    off = torch.tensor([0, last // 3, last // 3, last], dtype=torch.int32, device="cuda")
    out = torch.full((R, N), float("nan"), dtype=out_dtype, device="cuda")
    qm.grouped_gemm_fp8(a, a_s, w, w_s, off, out=out)
    want, bound = grouped_ref(a[:last], a_s[:last], w, w_s, off, torch.arange(last, device="cuda"), out_dtype == BF16)
    R8.check_rounded(out[:last], want, bound, out_dtype)
    assert (out[last:] == 0).all()


@pytest.mark.parametrize("R", [10, 700])
def test_grouped_clamps_offsets_and_rows(R):
    """Offsets and perm that no dispatch writes are clamped, never followed:
    the rows that sound ranges cover are right."""
    E, N, K, T = 3, 64, 128, 4
    g = gen(R)
    a, a_s, w, w_s = R8.codes(g, T, K), R8.scales(g, T, 1), R8.codes(g, E, N, K), R8.scales(g, E, 1, 1)
    off = torch.tensor([-5, 6, 4, 1 << 30], dtype=torch.int32, device="cuda")     # rows [0,6), none, [4,R)
    perm = torch.randint(-(1 << 31), (1 << 31) - 1, (R,), generator=g, device="cuda").to(torch.int32)
    src = torch.clamp(torch.div(perm.long(), 2, rounding_mode="trunc"), 0, T - 1)
    out = qm.grouped_gemm_fp8(a, a_s, w, w_s, off, perm=perm, k=2)
    ok = [(0, slice(0, 4)), (2, slice(6, R))]          # rows 4 and 5 are claimed twice
    for e, r in ok:
        want, bound = R8.product(a[src[r]], a_s[src[r]], w[e], w_s[e])
        R8.check_rounded(out[r], want, bound, F32)


@pytest.mark.parametrize("d,f", [(128, 128), (416, 288), (96, 32)])
@pytest.mark.parametrize("T,E,k,only", ROUTES)
def test_gate_up(T, E, k, only, d, f):
    g = gen(T + E + k + d)
    off, perm, _ = R8.routing(g, T, E, k, only=only)
    a, a_s = R8.codes(g, T, d), R8.scales(g, T, runs(d), mean=2.0 ** -6)
    mats = [m for _ in range(2) for m in (R8.codes(g, E, f, d), R8.scales(g, E, runs(f), runs(d), mean=2.0 ** -9))]
    q, sc = qm.expert_gate_up_fp8(a, a_s, *mats, off, perm, k)
    o, src = off.tolist(), perm.long() // k
    for e in range(E):
        r = slice(o[e], o[e + 1])
        if o[e + 1] > o[e]:
            v, dv = R8.gate_up(a[src[r]], a_s[src[r]], *(m[e] for m in mats))
            R8.check_quantised(q[r], sc[r], v, dv, f"expert {e}")


WIDE = [  # T, E, k, only, d, f: workgroups of whole runs, with 1 to 128 and more rows of an expert
    (200, 16, 4, None, 160, 2080), (40, 64, 1, None, 96, 1152), (90, 8, 1, [3], 288, 6400), (700, 2, 1, None, 128, 5152),
    (1, 1, 1, None, 4096, 96), (3, 2, 2, None, 2080, 288), (33, 1, 1, None, 3200, 1056), (600, 4, 1, [0, 1], 416, 2048)]


@pytest.mark.parametrize("T,E,k,only,d,f", WIDE)
def test_gate_up_wide(T, E, k, only, d, f):
    test_gate_up(T, E, k, only, d, f)


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("T,E,k,only,K,N", WIDE)
def test_grouped_gemm_wide(T, E, k, only, K, N, out_dtype):
    test_grouped_gemm(T, E, k, only, 2 * N + 1, K, out_dtype)


@pytest.mark.parametrize("T", [9, 150, 513, 3000])
def test_gate_up_of_overlapping_offsets_stays_in_its_buffers(T):
    """Offsets that claim rows many times over make more runs of rows than any
    sound ones: nothing is written past the workspace or the outputs."""
    E, k, d, f = 7, 2, 256, 288
    g = gen(T)
    R, NB = T * k, 3
    a, a_s = R8.codes(g, T, d), R8.scales(g, T, 2)
    gate, up = R8.codes(g, E, f, d), R8.codes(g, E, f, d)
    gs, us = R8.scales(g, E, NB, 2), R8.scales(g, E, NB, 2)
    off = torch.tensor([0, R, 0, R, 0, R, 0, R], dtype=torch.int32, device="cuda")
    perm = torch.arange(R, device="cuda").to(torch.int32)
    n = qm.lib().moe_expert_gate_up_fp8_workspace_bytes(ctypes.byref(qm.moe_shape(T, d, E, k, f)))
    guard = 4096
    ws = torch.full((n + guard,), 0xA5, dtype=torch.uint8, device="cuda")
    act = torch.full((R * f + guard,), 0xA5, dtype=torch.uint8, device="cuda")
    sc = torch.full((R * NB + guard,), -3.0, device="cuda")
    qm.expert_gate_up_fp8(a, a_s, gate, gs, up, us, off, perm, k, act=act[:R * f].view(R, f),
                          act_scales=sc[:R * NB].view(R, NB), ws=ws[:n] if n else None)
    assert (ws[n:] == 0xA5).all() and (act[R * f:] == 0xA5).all() and (sc[R * NB:] == -3.0).all()


@pytest.mark.parametrize("T", [6, 400])
def test_gate_up_leaves_rows_past_the_last_expert(T):
    E, k, d, f = 4, 2, 160, 160
    g = gen(T)
    a, a_s = R8.codes(g, T, d), R8.scales(g, T, 2)
    mats = [m for _ in range(2) for m in (R8.codes(g, E, f, d), R8.scales(g, E, 2, 2))]
    last = T
    off = torch.tensor([0, 0, last // 2, last // 2, last], dtype=torch.int32, device="cuda")
    perm = torch.arange(T * k, dtype=torch.int32, device="cuda")
    act = torch.full((T * k, f), 0x55, dtype=torch.uint8, device="cuda")
    sc = torch.full((T * k, 2), 9.0, device="cuda")
    qm.expert_gate_up_fp8(a, a_s, *mats, off, perm, k, act=act, act_scales=sc)
    assert (act[last:] == 0x55).all() and (sc[last:] == 9).all() and (sc[:last] != 9).all()


# ------------------------------------------------------- together, and reuse

def layer_case(T, d, E, k, f, seed=0):
    g = gen(seed)
    x = torch.randn((T, d), generator=g, device="cuda")
    res = torch.randn((T, d), generator=g, device="cuda").to(BF16)
    w = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(BF16)
    wr = torch.randn((E, d), generator=g, device="cuda") / d ** 0.5
    bias = torch.randn(E, generator=g, device="cuda")
    ex = qm.ExpertsFp8(R8.codes(g, E, f, d), R8.scales(g, E, runs(f), runs(d), mean=1 / (112 * d ** 0.5)),
                       R8.codes(g, E, f, d), R8.scales(g, E, runs(f), runs(d), mean=1 / (112 * d ** 0.5)),
                       R8.codes(g, E, d, f), R8.scales(g, E, runs(d), runs(f), mean=1 / (112 * f ** 0.5)))
    return x, res, w, wr, bias, ex


SHAPES = [(1, 512, 8, 2, 256), (5, 256, 64, 2, 160), (16, 128, 8, 4, 128), (100, 288, 4, 2, 416), (700, 512, 8, 2, 384)]


@pytest.mark.parametrize("T,d,E,k,f", SHAPES)
def test_layer_is_its_calls_in_sequence(T, d, E, k, f):
    x, res, w, wr, bias, ex = layer_case(T, d, E, k, f)
    y, h, q, sc = qm.add_rmsnorm(x, w, residual=res, fp8=True)
    out, ids, tw, logits = qm.layer_fp8(y, q, sc, ex, k, w_router=wr, bias=bias, check=True)
    # the calls
    s = qm.Shape(T, d, E, k, f)
    ws = qm.alloc_workspace(s)
    lg, ids2 = torch.empty_like(logits), torch.empty_like(ids)
    tw2 = torch.empty_like(tw)
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    perm, inv = (torch.empty(T * k, dtype=torch.int32, device="cuda") for _ in range(2))
    qm.moe_route_topk(s, y, wr, bias, lg, ids2, tw2)
    qm.moe_dispatch(s, ids2, off, perm, inv, ws)
    act, acts = qm.expert_gate_up_fp8(q, sc, ex.gate, ex.gate_scales, ex.up, ex.up_scales, off, perm, k)
    yy = qm.grouped_gemm_fp8(act, acts, ex.down, ex.down_scales, off)
    out2 = torch.empty_like(out)
    qm.moe_combine(s, yy, inv, tw2, out2)
    assert torch.equal(ids, ids2) and torch.equal(tw, tw2) and torch.equal(logits, lg) and torch.equal(out, out2)
    # and float64 from the device's own act (its codes are checked above)
    o, want = off.tolist(), torch.zeros((T * k, d), dtype=torch.float64, device="cuda")
    for e in range(E):
        if o[e + 1] > o[e]:
            r = slice(o[e], o[e + 1])
            want[r], _ = R8.product(act[r], acts[r], ex.down[e], ex.down_scales[e])
    full = (want[inv.long()].view(T, k, d) * tw.double()[..., None]).sum(1)
    assert (out.double() - full).norm() <= 1e-6 * full.norm()


def run_chain(x, res, w, wr, bias, ex, k, ws, stream=None):
    y, h, q, sc = qm.add_rmsnorm(x, w, residual=res, fp8=True, stream=stream)
    out, ids, tw, _ = qm.layer_fp8(y, q, sc, ex, k, w_router=wr, bias=bias, ws=ws, stream=stream)
    dense = qm.gemm_fp8(q, sc, ex.gate[0], ex.gate_scales[0], stream=stream)
    return h, out, ids, tw, dense


@pytest.mark.parametrize("T,d,E,k,f", SHAPES)
def test_chain_captured_and_replayed(T, d, E, k, f):
    x, res, w, wr, bias, ex = layer_case(T, d, E, k, f)
    s = qm.Shape(T, d, E, k, f)
    eager_ws, ws = qm.alloc_workspace_fp8(s), qm.alloc_workspace_fp8(s)
    run_chain(x, res, w, wr, bias, ex, k, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run_chain(x, res, w, wr, bias, ex, k, ws)
    for i in range(4):
        x.copy_(torch.randn((T, d), generator=gen(50 + i), device="cuda"))
        want = [t.clone() for t in run_chain(x, res, w, wr, bias, ex, k, eager_ws)]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_captured_graphs_share_a_workspace():
    cases = [layer_case(T, 256, 8, 2, 256, seed=T) for T in (9, 300)]
    shapes = [qm.Shape(T=c[0].shape[0], d=256, E=8, k=2, f=256) for c in cases]
    ws = max((qm.alloc_workspace_fp8(s) for s in shapes), key=lambda t: t.numel())
    want = [[t.clone() for t in run_chain(*c, 2, None)] for c in cases]
    graphs, got = [], []
    for c in cases:
        run_chain(*c, 2, ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(run_chain(*c, 2, ws))
        graphs.append(graph)
    for order in ((0, 1), (1, 0), (0, 0, 1, 1)):
        for ts in got:
            for t in ts:
                t.zero_()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for g_, w_ in zip(got, want):
            for p, q in zip(g_, w_):
                assert torch.equal(p, q)


def test_two_streams_at_once():
    a, b = layer_case(300, 256, 8, 2, 256, seed=1), layer_case(7, 256, 8, 2, 256, seed=2)
    want = [run_chain(*c, 2, None) for c in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [run_chain(*c, 2, None, stream=st) for c, st in zip((a, b), streams)]
        torch.cuda.synchronize()
        for g_, w_ in zip(got, want):
            for p, q in zip(g_, w_):
                assert torch.equal(p, q)


# ------------------------------------------------- offsets beyond 32 bits

@pytest.mark.parametrize("R", [3, 300, 5000])
def test_grouped_weights_beyond_4_gib(R):
    E, N, K = 33, 8192, 16384
    g = gen(R)
    w = torch.zeros((E, N, K), dtype=torch.uint8, device="cuda")
    w[-1] = R8.codes(g, N, K).view(torch.uint8)
    w_s = torch.zeros((E, N // 128, K // 128), device="cuda")
    w_s[-1] = R8.scales(g, N // 128, K // 128)
    a, a_s = R8.codes(g, R, K), R8.scales(g, R, K // 128)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = R
    out = qm.grouped_gemm_fp8(a, a_s, w, w_s, off)
    assert torch.equal(out, qm.grouped_gemm_fp8(a, a_s, w[-1:], w_s[-1:], off[-2:]))
    want, bound = R8.product(a[-3:], a_s[-3:], w[-1].view(torch.float8_e4m3fn), w_s[-1])
    R8.check_rounded(out[-3:], want, bound, F32)
    act, act_s = qm.expert_gate_up_fp8(a, a_s, w, w_s, w, w_s, off, torch.arange(R, device="cuda").to(torch.int32), 1)
    one = qm.expert_gate_up_fp8(a, a_s, w[-1:], w_s[-1:], w[-1:], w_s[-1:], off[-2:],
                                torch.arange(R, device="cuda").to(torch.int32), 1)
    assert torch.equal(act.view(torch.uint8), one[0].view(torch.uint8)) and torch.equal(act_s, one[1])


@pytest.mark.parametrize("M", [20, 600])
def test_gemm_rows_and_outputs_beyond_32_bits(M):
    N, K = 160, 256
    a, a_s, w, w_s = gemm_case(M, N, K)
    step = (5 << 30) // M // 64 * 64
    rows = torch.zeros(M * step, dtype=torch.uint8, device="cuda").as_strided((M, K), (step, 1))
    rows.copy_(a.view(torch.uint8))
    for dt in (F32, BF16):
        out = torch.zeros(M * step, dtype=dt, device="cuda").as_strided((M, N), (step, 1))
        qm.gemm_fp8(rows, a_s, w, w_s, out=out)
        assert torch.equal(out, qm.gemm_fp8(a, a_s, w, w_s, out_dtype=dt))


def test_norm_rows_beyond_32_bits():
    T, d = 40, 4096
    x, res, w = norm_case(T, d, F32, BF16, BF16)
    step = (5 << 30) // T // 64 * 64
    far = lambda t: torch.zeros(T * step, dtype=t.dtype, device="cuda").as_strided((T, d), (step, 1)).copy_(t)  # noqa: E731
    want = qm.add_rmsnorm(x, w, residual=res, fp8=True)
    out = far(torch.zeros_like(res))
    got = qm.add_rmsnorm(far(x), w, residual=far(res), residual_out=out, fp8=True)
    for p, q in zip(got, want):
        assert torch.equal(p.contiguous().view(torch.uint8), q.view(torch.uint8))


def test_python_refusals():
    a, a_s, w, w_s = gemm_case(4, 64, 256)
    for bad in (lambda: qm.gemm_fp8(a, a_s[:, :1].contiguous(), w, w_s), lambda: qm.gemm_fp8(a, a_s, w[:, :128], w_s),
                lambda: qm.gemm_fp8(a.float(), a_s, w, w_s), lambda: qm.gemm_fp8(a, a_s.double(), w, w_s),
                lambda: qm.gemm_fp8(a, a_s, w, w_s, out_dtype=torch.float16),
                lambda: qm.gemm_fp8(a, a_s, w, w_s, out=torch.empty((4, 65), device="cuda")),
                lambda: qm.gemm_fp8(a.t(), a_s, w, w_s), lambda: qm.gemm_fp8(a, a_s.cpu(), w, w_s),
                lambda: qm.grouped_gemm_fp8(a, a_s, w[None], w_s[None], torch.zeros(3, dtype=torch.int32, device="cuda")),
                lambda: qm.grouped_gemm_fp8(a, a_s, w[None], w_s[None], torch.zeros(2, dtype=torch.int64, device="cuda")),
                lambda: qm.add_rmsnorm(a_s, a_s[0]), lambda: qm.add_rmsnorm(a_s.double()),
                lambda: qm.add_rmsnorm(a_s, residual=a_s[:2]), lambda: qm.add_rmsnorm(a_s, residual_out=a_s)):
        with pytest.raises((ValueError, qm.MoeError)):
            bad()
