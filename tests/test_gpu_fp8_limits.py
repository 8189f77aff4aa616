"""The FP8 operators on the GPU where their documentation allows a call that
sums, sizes or buffers of the ordinary tests do not reach."""

import pytest
import torch

import fp8_ref as R8
import quantized_routed_moe_amd as qm
from fp8_ref import gen, runs

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


# ------------------------------------- steps whose large products cancel

def cancelling(g, rows_a, rows_w, K):
    """Codes whose step of 128 holds two products of +-448^2 that cancel, at
    places that differ from step to step, and positive products of 0.25 to 4
    besides: an evaluation that drops what lies 16 bits below the largest
    product loses all but the large ones."""
    a = torch.exp2(2 * torch.rand((rows_a, K), generator=g, device="cuda") - 1)
    w = torch.exp2(2 * torch.rand((rows_w, K), generator=g, device="cuda") - 1)
    for s in range(runs(K)):
        i, j = 128 * s + s % 32, 128 * s + 31 - (3 * s) % 16
        a[:, i], a[:, j], w[:, i], w[:, j] = 448.0, 448.0, 448.0, -448.0
    return a.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn)


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K", [(5, 512, 320), (70, 512, 1024), (600, 512, 320), (600, 512, 1024), (5000, 1111, 512)])
def test_gemm_sums_in_32_bits_where_products_cancel(M, N, K, out_dtype):
    """Both result types, whatever the number of rows: fp32 sums (their bound,
    136 roundings of a step's magnitudes, is about 3 here, the sum about 200)
    and one rounding to the result's type."""
    g = gen(M + K)
    a, w = cancelling(g, M, N, K)
    a_s, w_s = R8.scales(g, M, runs(K)), R8.scales(g, runs(N), runs(K))
    want, bound = R8.product(a, a_s, w, w_s)
    R8.check_rounded(qm.gemm_fp8(a, a_s, w, w_s, out_dtype=out_dtype), want, bound, out_dtype)


@pytest.mark.parametrize("R", [40, 2400, 9000])
def test_grouped_bf16_sums_in_32_bits_where_products_cancel(R):
    g = gen(R)
    E, N, K = 4, 600, 384
    mats = [cancelling(g, R if e == 0 else 1, N, K) for e in range(E)]
    a, w = mats[0][0], torch.stack([m[1] for m in mats])
    a_s, w_s = R8.scales(g, R, runs(K)), R8.scales(g, E, runs(N), runs(K))
    off = [0, R // 3, R // 3, R // 2, R]
    out = qm.grouped_gemm_fp8(a, a_s, w, w_s, torch.tensor(off, dtype=torch.int32, device="cuda"), out_dtype=BF16)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        if off[e + 1] > off[e]:
            want, bound = R8.product(a[r], a_s[r], w[e], w_s[e])
            R8.check_rounded(out[r], want, bound, BF16, f"expert {e}")


# ----------------------------------------------------- the layer's routing

def layer_case(T, d, E, k, f, seed=0):
    g = gen(seed)
    q, sc = R8.codes(g, T, d), R8.scales(g, T, runs(d), mean=2.0 ** -8)
    ex = qm.ExpertsFp8(R8.codes(g, E, f, d), R8.scales(g, E, runs(f), runs(d), mean=1 / (112 * d ** 0.5)),
                       R8.codes(g, E, f, d), R8.scales(g, E, runs(f), runs(d), mean=1 / (112 * d ** 0.5)),
                       R8.codes(g, E, d, f), R8.scales(g, E, runs(d), runs(f), mean=1 / (112 * f ** 0.5)))
    return q, sc, ex, torch.randn((T, E), generator=g, device="cuda")


@pytest.mark.parametrize("T,d,E,k,f", [(1, 512, 8, 2, 256), (30, 256, 64, 3, 160), (700, 288, 8, 2, 384)])
def test_layer_of_given_logits(T, d, E, k, f):
    """No router weights and no x: the layer routes on the logits it is given,
    and leaves them as they were."""
    q, sc, ex, lg = layer_case(T, d, E, k, f, seed=T)
    given = lg.clone()
    out, ids, tw, back = qm.layer_fp8(None, q, sc, ex, k, logits=lg, check=True)
    assert back is lg and torch.equal(lg, given)
    assert torch.equal(ids.long(), lg.topk(k, dim=1).indices)
    want_w = torch.softmax(lg.double().topk(k, dim=1).values, 1)
    assert ((tw.double() - want_w).abs() <= 8 * R8.U32).all()      # exp, sum, division: values up to 1
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    perm, inv = (torch.empty(T * k, dtype=torch.int32, device="cuda") for _ in range(2))
    s = qm.Shape(T, d, E, k, f)
    qm.moe_dispatch(s, ids, off, perm, inv, qm.alloc_workspace(s))
    act, acts = qm.expert_gate_up_fp8(q, sc, ex.gate, ex.gate_scales, ex.up, ex.up_scales, off, perm, k)
    want = torch.empty_like(out)
    qm.moe_combine(s, qm.grouped_gemm_fp8(act, acts, ex.down, ex.down_scales, off), inv, tw, want)
    assert torch.equal(out, want)


def test_layer_refuses_missing_and_misplaced_logits():
    q, sc, ex, lg = layer_case(4, 256, 8, 2, 128)
    for bad in (dict(), dict(logits=lg[:, :7].contiguous()), dict(logits=lg.double()), dict(logits=lg.cpu()),
                dict(w_router=torch.zeros((8, 256), device="cuda")), dict(logits=lg, bias=lg[0])):
        with pytest.raises((ValueError, qm.MoeError)):
            qm.layer_fp8(None, q, sc, ex, 2, **bad)


def test_workspace_belongs_to_its_stream():
    """A freed workspace of a stream is not handed to an allocation of another
    stream, in which its last kernels may still be running."""
    s = qm.Shape(300, 512, 8, 2, 512)
    side = torch.cuda.Stream()
    torch.cuda.empty_cache()
    ws = qm.alloc_workspace_fp8(s, stream=side)
    side.synchronize()
    assert (ws[:256] == 0).all()
    at, n = ws.data_ptr(), ws.numel()
    del ws
    other = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert other.data_ptr() != at
    with torch.cuda.stream(side):
        again = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert again.data_ptr() == at
    q, sc, ex, lg = layer_case(300, 512, 8, 2, 512)
    want = qm.layer_fp8(None, q, sc, ex, 2, logits=lg)
    torch.cuda.synchronize()
    got = qm.layer_fp8(None, q, sc, ex, 2, logits=lg, ws=qm.alloc_workspace_fp8(s, stream=side), stream=side, check=True)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


# --------------------------------------------- more rows than one grid holds

@pytest.mark.parametrize("T", [(1 << 23) + 3, (1 << 24) + 5])
def test_norm_of_more_rows_than_a_grid_holds(T):
    """Rows of 32: at 256 threads a row, 2^24 of them are as many threads as
    no grid has.  Every row against float64, in parts."""
    d = 32
    g = gen(T)
    x = torch.randn((T, d), generator=g, device="cuda")
    res = torch.randn((T, d), generator=g, device="cuda").to(BF16)
    w = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(BF16)
    y, h, q, sc = qm.add_rmsnorm(x, w, residual=res, fp8=True)
    for t in range(0, T, 1 << 21):
        r = slice(t, t + (1 << 21))
        want_h, v, dv = R8.norm(x[r], res[r], w, 1e-6)
        assert torch.equal(h[r], want_h)
        R8.check_rounded(y[r], v, dv, BF16, f"y from row {t}")
        R8.check_quantised(q[r], sc[r], v, dv, f"q from row {t}")


def test_norm_of_many_rows_in_place_and_from_one_row():
    """The rows of the second launch: one row of x for all, a residual taken
    in place with other values between its rows, no E4M3 output."""
    T, d = (1 << 23) + 9, 32
    g = gen(5)
    x = torch.randn((1, d), generator=g, device="cuda")
    buf = torch.randn((T, d + 8), generator=g, device="cuda").to(BF16)
    want = (x + buf[:, :d].float()).to(BF16)
    rest = buf[:, d:].clone()
    y, h, _, _ = qm.add_rmsnorm(x.expand(T, d), None, residual=buf[:, :d], residual_out=buf[:, :d])
    assert torch.equal(buf[:, :d], want) and torch.equal(buf[:, d:], rest)
    _, v, dv = R8.norm(want[-64:], None, None, 1e-6)
    R8.check_rounded(y[-64:], v, dv, BF16)


# ------------------------------------------------- wide products of few rows

def time_of(call, n=10):
    """Least time of a pass, in us, of n passes in a replayed graph."""
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(n):
            call()
    best = float("inf")
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3 / n)
    return best


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("M", [1, 16, 17, 40, 130, 300, 600, 900])
@pytest.mark.parametrize("N", [12300, 84731, 84736 + 256])
def test_gemm_wide(M, N, out_dtype):
    """Column tiles in numbers that four and eight do not divide, of one to
    several runs of rows."""
    K = 160
    g = gen(M + N)
    a, a_s, w, w_s = R8.codes(g, M, K), R8.scales(g, M, 2), R8.codes(g, N, K), R8.scales(g, runs(N), 2)
    want, bound = R8.product(a, a_s, w, w_s)
    R8.check_rounded(qm.gemm_fp8(a, a_s, w, w_s, out_dtype=out_dtype), want, bound, out_dtype)


def test_gemm_of_an_odd_number_of_tiles_uses_the_whole_chip():
    """501 column tiles take about as long as 504; left to one XCD of eight
    they took three times as long."""
    M, K, us = 17, 4096, []
    g = gen(1)
    a, a_s = R8.codes(g, M, K), R8.scales(g, M, 32)
    for N in (501 * 256, 504 * 256):
        w, w_s = R8.codes(g, N, K), R8.scales(g, 2 * N // 256, 32)
        us.append(time_of(lambda: qm.gemm_fp8(a, a_s, w, w_s)))
    assert us[0] < 1.5 * us[1], us


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("M", [1, 4])
def test_gemm_of_few_rows_does_not_depend_on_the_columns(M, out_dtype):
    """Up to four rows: a column's sum is the same bits in a product of 256
    columns and of 90000, on one kernel whatever the columns."""
    N, K = 90000, 4096
    g = gen(2)
    a, a_s, w, w_s = R8.codes(g, M, K), R8.scales(g, M, 32), R8.codes(g, N, K), R8.scales(g, runs(N), 32)
    wide = qm.gemm_fp8(a, a_s, w, w_s, out_dtype=out_dtype)
    for n in (0, 1 << 14, 1 << 16):
        few = qm.gemm_fp8(a, a_s, w[n:n + 256], w_s[n // 128:n // 128 + 2], out_dtype=out_dtype)
        assert torch.equal(wide[:, n:n + 256], few)


def test_grouped_gemm_of_more_columns_than_few_row_workgroups_fit():
    """A row or two an expert of 2^21 columns: more workgroups of 16 columns
    than a grid holds."""
    E, N, K, R = 64, (1 << 21) - 48, 32, 100
    g = gen(7)
    w = torch.randint(0, 120, (E, N, K), generator=g, device="cuda", dtype=torch.uint8)       # codes of 0 to 256
    a, a_s, w_s = R8.codes(g, R, K), R8.scales(g, R, 1), R8.scales(g, E, runs(N), 1)
    off = torch.linspace(0, R, E + 1, device="cuda").to(torch.int32)
    out = qm.grouped_gemm_fp8(a, a_s, w, w_s, off)
    o = off.tolist()
    for e in range(E):
        r = slice(o[e], o[e + 1])
        for n in (0, 1 << 20, N - 300):
            n -= n % 128
            c = slice(n, min(n + 300, N))
            want, bound = R8.product(a[r], a_s[r], w[e, c].view(torch.float8_e4m3fn), w_s[e, n // 128:runs(c.stop)])
            R8.check_rounded(out[r, c], want, bound, F32)


# ---------------------------------------------- rows past the last expert

@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("R,E,N,off", [
    (1, 1, 50, [0, 0]), (9, 8, 271, [0, 0, 1, 1, 2, 2, 3, 4, 8]), (70, 64, 272, [0] + [1] * 64), (40, 2, 30, [0, 20, 39]),
    (129, 1, 4096, [0, 1]), (700, 3, 1111, [0, 100, 101, 573]), (5000, 4, 1024, [0, 0, 64, 64, 129]),
    (5000, 64, 4100, [0] + [i for i in range(64)]), (20000, 5, 2048, [0] * 6), (3000, 2, 77, [0, 1500, 2999])])
def test_grouped_zeroes_rows_past_the_last_expert(R, E, N, off, out_dtype):
    """On every path, rows that end inside a run, columns that end inside a
    tile, and nothing behind the last row."""
    K = 96
    g = gen(R + N)
    a, a_s, w, w_s = R8.codes(g, R, K), R8.scales(g, R, 1), R8.codes(g, E, N, K), R8.scales(g, E, runs(N), 1)
    buf = torch.full((R * N + 4096,), 7.0, dtype=out_dtype, device="cuda")
    out = buf[:R * N].view(R, N)
    qm.grouped_gemm_fp8(a, a_s, w, w_s, torch.tensor(off, dtype=torch.int32, device="cuda"), out=out)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        if off[e + 1] > off[e]:
            want, bound = R8.product(a[r], a_s[r], w[e], w_s[e])
            R8.check_rounded(out[r], want, bound, out_dtype, f"expert {e}")
    assert (out[off[-1]:] == 0).all() and (buf[R * N:] == 7).all()


def test_grouped_time_of_rows_past_the_last_expert():
    """64 live rows of 16384: about the time that zeros take (and less than
    four times it), not the time of one workgroup that writes them in turn."""
    R, E, N, K = 16384, 8, 4096, 256
    g = gen(3)
    a, a_s, w, w_s = R8.codes(g, R, K), R8.scales(g, R, 2), R8.codes(g, E, N, K), R8.scales(g, E, runs(N), 2)
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda") * 8
    out = torch.empty((R, N), device="cuda")
    us = [time_of(lambda: qm.grouped_gemm_fp8(a, a_s, w, w_s, off, out=out)), time_of(lambda: out.zero_())]
    assert us[0] < 4 * us[1], us


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("R,N,off", [(9, 271, [4, 6, 8]), (1, 40, [1, 1]), (600, 1111, [130, 130, 300, 599]),
                                     (5000, 1024, [4000, 4100, 5000]), (5000, 1024, [129, 129, 260]), (300, 64, [300] * 3)])
def test_grouped_rows_below_the_first_offset_are_zero(R, N, off, out_dtype):
    """The experts of one part of a dispatch: offsets that do not begin at 0."""
    E, K = len(off) - 1, 160
    g = gen(R + N)
    a, a_s, w, w_s = R8.codes(g, R, K), R8.scales(g, R, 2), R8.codes(g, E, N, K), R8.scales(g, E, runs(N), 2)
    out = torch.full((R, N), float("nan"), dtype=out_dtype, device="cuda")
    qm.grouped_gemm_fp8(a, a_s, w, w_s, torch.tensor(off, dtype=torch.int32, device="cuda"), out=out)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        if off[e + 1] > off[e]:
            want, bound = R8.product(a[r], a_s[r], w[e], w_s[e])
            R8.check_rounded(out[r], want, bound, out_dtype, f"expert {e}")
    assert (out[:off[0]] == 0).all() and (out[off[-1]:] == 0).all()


# ------------------------------------- non-finite values of gate/up's output

GATE_UP_PATHS = [(3, 2, 1, 256), (100, 8, 2, 1056), (900, 4, 2, 2048)]      # T, E, k, f: 16, 32 and 128 columns a workgroup


@pytest.mark.parametrize("T,E,k,f", GATE_UP_PATHS)
def test_gate_up_of_nan_codes(T, E, k, f):
    """A NaN in a token makes its rows NaN, one in a weight row that column of
    the expert; a NaN does not enter its run's maximum, so every other code
    and scale is what it is without that column."""
    d = 160
    g = gen(T)
    off, perm, _ = R8.routing(g, T, E, k)
    a, a_s = R8.codes(g, T, d), R8.scales(g, T, 2, mean=2.0 ** -6)
    gate, up = R8.codes(g, E, f, d), R8.codes(g, E, f, d)
    gs, us = R8.scales(g, E, runs(f), 2), R8.scales(g, E, runs(f), 2)
    ua, ug, uu = (t.view(torch.uint8).clone() for t in (a, gate, up))
    bad = T // 2
    n0, n1 = f - 20, 37
    uu0 = uu.clone()
    uu0[:, n0] = 0                       # v = 0 there: does not enter the maximum either
    uu0[:, n1] = 0
    want, want_s = qm.expert_gate_up_fp8(ua, a_s, ug, gs, uu0, us, off, perm, k)
    ua[bad, 159], ug[:, n0, 3], uu[:, n1, 131] = 0x7F, 0xFF, 0x7F
    q, sc = qm.expert_gate_up_fp8(ua, a_s, ug, gs, uu, us, off, perm, k)
    q, want = q.view(torch.float8_e4m3fn).float(), want.view(torch.float8_e4m3fn).float()
    rows = perm.long() // k == bad
    assert rows.sum() == k and torch.isnan(q[rows]).all() and (sc[rows] == R8.SCALE_MIN).all()
    col = torch.zeros(f, dtype=torch.bool, device="cuda")
    col[n0] = col[n1] = True
    assert torch.isnan(q[:, col]).all()
    assert torch.equal(q[~rows][:, ~col], want[~rows][:, ~col]) and torch.equal(sc[~rows], want_s[~rows])


@pytest.mark.parametrize("T,E,k,f", GATE_UP_PATHS)
def test_gate_up_of_overflowing_values(T, E, k, f):
    """up overflows to an infinity in one column of a run whose other values
    are 0: scale infinite, code NaN there and 0 beside it; the other runs are
    not touched."""
    d = 128
    g = gen(T + 1)
    off, perm, _ = R8.routing(g, T, E, k)
    a, a_s = R8.codes(g, T, d).float().abs().add(16).clamp(max=448).to(torch.float8_e4m3fn), torch.full((T, 1), 2.0 ** -6, device="cuda")
    gate, up = (R8.codes(g, E, f, d).float().abs().add(16).clamp(max=448).to(torch.float8_e4m3fn) for _ in range(2))
    gs, us = (torch.full((E, runs(f), 1), 2.0 ** -9, device="cuda") for _ in range(2))
    want, want_s = qm.expert_gate_up_fp8(a, a_s, gate, gs, up, us, off, perm, k)
    b, n = 1, 128 + 77
    uu = up.view(torch.uint8).clone()
    uu[:, 128:256] = 0
    uu[:, n] = up.view(torch.uint8)[:, n]
    us[:, b] = 3e38
    q, sc = qm.expert_gate_up_fp8(a, a_s, gate, gs, uu, us, off, perm, k)
    qf, wf = q.float(), want.float()
    assert torch.isinf(sc[:, b]).all() and torch.isnan(qf[:, n]).all()
    run = torch.zeros(f, dtype=torch.bool, device="cuda")
    run[128:256] = True
    others = run.clone()
    others[n] = False
    assert (qf[:, others] == 0).all()
    assert torch.equal(qf[:, ~run], wf[:, ~run])
    keep = torch.arange(sc.shape[1], device="cuda") != b
    assert torch.equal(sc[:, keep], want_s[:, keep])


# ------------------------------------------ a layer of 2^24 tokens and more

def test_layer_of_more_tokens_than_a_grid_of_256_threads_holds():
    T, d, E, k, f = (1 << 24) + 3, 32, 2, 1, 32
    q, sc, ex, lg = layer_case(T, d, E, k, f, seed=11)
    out, ids, tw, _ = qm.layer_fp8(None, q, sc, ex, k, logits=lg, check=True)
    assert torch.equal(ids[:, 0].long(), lg.argmax(1)) and (tw == 1).all()
    perm = torch.sort(ids[:, 0].long(), stable=True).indices
    off = torch.cat([ids.new_zeros(1), torch.bincount(ids[:, 0].long(), minlength=E).cumsum(0).to(torch.int32)])
    act, acts = qm.expert_gate_up_fp8(q, sc, ex.gate, ex.gate_scales, ex.up, ex.up_scales, off, perm.to(torch.int32), k)
    y = qm.grouped_gemm_fp8(act, acts, ex.down, ex.down_scales, off)
    want = torch.empty_like(y)
    want[perm] = y
    assert torch.equal(out, want)


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("R,N,K", [(1, 4096, 2048), (4, 4096, 2048), (16, 4096, 1024), (40, 4096, 2048), (500, 1024, 512)])
def test_grouped_of_one_expert_is_the_dense_product(R, N, K, out_dtype):
    """The same kernel and the same order of sums: items that could hold rows
    of no expert change nothing."""
    g = gen(R)
    a, a_s, w, w_s = R8.codes(g, R, K), R8.scales(g, R, runs(K)), R8.codes(g, N, K), R8.scales(g, runs(N), runs(K))
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    got = qm.grouped_gemm_fp8(a, a_s, w[None], w_s[None], off, out_dtype=out_dtype)
    assert torch.equal(got, qm.gemm_fp8(a, a_s, w, w_s, out_dtype=out_dtype))
