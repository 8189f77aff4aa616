"""The operators of a batch of many requests as they are used: together in a
step, captured and replayed, on streams of their own, at once, with workspaces
that hold anything, behind offsets of more than 32 bits; and the sizes at which
they take another way."""

import math

import pytest
import torch

import batch_ref as B
import fp8_ref as R
import quantized_routed_moe_amd as qm
from batch_ref import gen

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def same(got, want):
    assert len(got) == len(want)
    for p, q in zip(got, want):
        assert (p is None and q is None) or torch.equal(p, q)


# ------------------------------------------------------- a step of a batch

class Step:
    """The end of a serving step: residual addition and norm, a projection in
    FP8 with each request's adapter on top, the vocabulary, the log
    probabilities of drafted tokens with alternatives."""

    def __init__(self, T, d, N, V, r, L, seed=0):
        g = gen(seed + T)
        self.x = torch.randn((T, d), generator=g, device="cuda").to(BF16)
        self.res = torch.randn((T, d), generator=g, device="cuda")
        self.ids = torch.randint(-1, L, (T,), generator=g, device="cuda", dtype=I32)
        self.tok = torch.randint(0, V, (T, 2), generator=g, device="cuda", dtype=I32)
        self.w, self.ws = R.codes(g, N, d), R.scales(g, R.runs(N), R.runs(d), mean=2.0 ** -7 / math.sqrt(d))
        self.vw, self.vs = R.codes(g, V, N), R.scales(g, R.runs(V), R.runs(N), mean=2.0 ** -6 / math.sqrt(N))
        self.a = (torch.randn((L, r, d), generator=g, device="cuda") / math.sqrt(d)).to(BF16)
        self.b = (torch.randn((L, N, r), generator=g, device="cuda") / math.sqrt(r)).to(BF16)
        self.s = torch.exp2(2 * torch.rand(L, generator=g, device="cuda") - 1)
        self.L = L
        lb = qm.lib()
        n = max(lb.moe_lora_add_workspace_bytes(T, d, N, r, L), lb.moe_token_logprobs_workspace_bytes(T, V, 6))
        self.ws_bytes = n

    def run(self, ws=None, stream=None):
        plan = qm.lora_plan(self.ids, self.L, stream=stream)
        y, _, q, sc = qm.add_rmsnorm(self.x, residual=self.res, fp8=True, stream=stream)
        h = qm.gemm_fp8(q, sc, self.w, self.ws, stream=stream)
        shared = h.clone() if stream is None else None
        qm.lora_add(h, y, self.a, self.b, plan, scales=self.s, out=h, ws=ws, stream=stream)
        _, _, q2, sc2 = qm.add_rmsnorm(h, y=False, fp8=True, stream=stream)
        logits = qm.gemm_fp8(q2, sc2, self.vw, self.vs, stream=stream)
        return (y, shared, h, logits, plan.perm, *qm.token_logprobs(logits, self.tok, top=6, entropy=True, ws=ws, stream=stream))


STEPS = [(1, 256, 512, 30011, 16, 3), (5, 512, 256, 20000, 32, 4), (70, 256, 320, 4099, 16, 9), (300, 512, 512, 2048, 72, 5)]


@pytest.mark.parametrize("T,d,N,V,r,L", STEPS)
def test_step(T, d, N, V, r, L):
    c = Step(T, d, N, V, r, L)
    y, shared, h, logits, perm, *out = c.run()
    want, bound = B.lora(shared, y, c.a, c.b, c.ids, c.s)
    B.check_rounded(h, want, bound, BF16)
    assert torch.isfinite(logits).all() and float(logits.float().std()) > 0.1
    B.check_scores(logits, c.tok, 6, out)


@pytest.mark.parametrize("T,d,N,V,r,L", STEPS)
def test_step_captured_and_replayed(T, d, N, V, r, L):
    """Other inputs, ids among them, in each replay; eager calls, of other
    sizes too, between them."""
    c, other = Step(T, d, N, V, r, L), Step(33, 256, 192, 9001, 24, 7)
    c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = c.run()
    for i in range(5):
        c.x.copy_(torch.randn((T, d), generator=gen(i), device="cuda"))
        c.ids.copy_(torch.randint(-1, L, (T,), generator=gen(90 + i), device="cuda", dtype=I32))
        want = [t.clone() for t in c.run()]
        other.run()
        graph.replay()
        if i % 2:
            other.run()
        torch.cuda.synchronize()
        same(got, want)


def test_two_captured_graphs_share_a_workspace():
    """One after the other, on one stream, and with what the workspace held
    before: nothing of it is taken for this call's."""
    cases = [Step(5, 512, 256, 20000, 32, 4), Step(70, 256, 320, 40000, 40, 9)]
    n = max(c.ws_bytes for c in cases)
    want = [[t.clone() for t in c.run()] for c in cases]
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    graphs, got = [], []
    for c in cases:
        c.run(ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(c.run(ws))
        graphs.append(graph)
    for order in ((0, 1), (1, 0), (0, 0, 1, 1)):
        for ts in got:
            for t in ts:
                t.zero_()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for g_, w_ in zip(got, want):
            same(g_, w_)
        ws.random_(0, 256)


@pytest.mark.parametrize("fill", [0, 0xff, None])
def test_workspaces_hold_anything(fill):
    c = Step(70, 512, 640, 30000, 72, 9)
    want = c.run()
    ws = torch.empty(c.ws_bytes, dtype=torch.uint8, device="cuda")
    for _ in range(4):
        ws.random_(0, 256) if fill is None else ws.fill_(fill)
        same(c.run(ws), want)
        same(c.run(ws), want)           # and its own of the call before


def test_two_streams_at_once():
    """Launches whose workgroups wait for others of theirs, side by side."""
    cases = [Step(300, 512, 2048, 5000, 72, 5), Step(64, 2048, 2048, 20000, 16, 64)]
    want = [c.run() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(6):
        got = [c.run(stream=st) for c, st in zip(cases, streams)]
        torch.cuda.synchronize()
        for g_, w_ in zip(got, want):
            same([t for i, t in enumerate(g_) if i != 1], [t for i, t in enumerate(w_) if i != 1])


# ------------------------------------------------------------------ sizes

@pytest.mark.parametrize("dtype,V", [(BF16, 1), (BF16, 63), (BF16, 700), (BF16, 4096), (F32, 5), (F32, 2048), (F32, 1023)])
@pytest.mark.parametrize("top", [0, 1, 5, 64])
@pytest.mark.parametrize("T", [2048, 2051])
def test_scores_of_many_short_rows(T, top, V, dtype):
    top = min(top, V)
    l = (2.5 * torch.randn((T, V), generator=gen(V + top), device="cuda")).to(dtype)
    l[::5] = l[::5].round()             # ties
    l[3::7] = 1.0                       # all equal: more at the bound than a list holds
    l[4::9, ::2] = -math.inf
    l[5::101] = -math.inf
    tok = torch.randint(0, V, (T, 1), generator=gen(1), device="cuda", dtype=I32)
    B.check_scores(l, tok, top, qm.token_logprobs(l, tok, top=top, entropy=True), f"T={T} V={V}")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("top", [3, 20])
def test_scores_of_many_long_rows(top, dtype):
    """A workgroup a row, over many rounds, ties and lists that overflow among them."""
    T, V = 1300, 20011
    l = (2.5 * torch.randn((T, V), generator=gen(top), device="cuda")).to(dtype)
    l[::5] = l[::5].round()
    l[3::7] = 1.0
    l[4::9, 1:] = -math.inf
    tok = torch.randint(0, V, (T,), generator=gen(1), device="cuda", dtype=I32)
    B.check_scores(l, tok, top, qm.token_logprobs(l, tok, top=top, entropy=True))


def test_scores_of_many_given_tokens():
    """As many as a call takes, the same ones again and again."""
    l = torch.randn((3, 5000), generator=gen(2), device="cuda")
    tok = torch.randint(0, 40, (3, 4096), generator=gen(3), device="cuda", dtype=I32)
    B.check_scores(l, tok, 0, qm.token_logprobs(l, tok))
    with pytest.raises(qm.MoeError):
        qm.token_logprobs(l, torch.zeros((3, 4097), dtype=I32, device="cuda"))


@pytest.mark.parametrize("K,r", [(4096, 16), (2080, 64), (4096, 128), (1056, 256)])
def test_lora_of_many_tokens(K, r):
    """Many halves, so that makers are dealt to XCDs, and as many that are empty."""
    T, N, L = 3001, 777, 40
    g = gen(r)
    x, a, b, base, s = B.lora_case(g, T, K, N, r, L, F32)
    ids = torch.randint(-1, L, (T // 60 + 1,), generator=g, device="cuda", dtype=I32).repeat_interleave(60)[:T].contiguous()
    got = qm.lora_add(base, x, a, b, qm.lora_plan(ids, L), scales=s)
    want, bound = B.lora(base, x, a, b, ids, s)
    B.check_rounded(got, want, bound, F32)


@pytest.mark.parametrize("r", [16, 32, 40])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5])
def test_lora_of_few_tokens(T, r):
    """With and without v handed over, tokens of one adapter and of several;
    the same call again gives the same bits."""
    K, N, L = 1184, 2055, 4
    for kind in ("one", "several"):
        g = gen(T + r)
        x, a, b, base, s = B.lora_case(g, T, K, N, r, L, BF16)
        ids = torch.full((T,), 2, dtype=I32, device="cuda") if kind == "one" else torch.arange(T, device="cuda", dtype=I32) % (L + 1)
        plan = qm.lora_plan(ids, L)
        got = qm.lora_add(base, x, a, b, plan, scales=s)
        want, bound = B.lora(base, x, a, b, ids, s)
        B.check_rounded(got, want, bound, BF16, kind)
        for _ in range(3):
            assert torch.equal(qm.lora_add(base, x, a, b, plan, scales=s), got)


@pytest.mark.parametrize("T", [1, 40])
def test_lora_of_non_finite_weights(T):
    """An infinity of b is in its column of its adapter's tokens only, one of
    base in its place."""
    K, N, r, L = 128, 130, 24, 3
    g = gen(T)
    x, a, b, base, s = B.lora_case(g, T, K, N, r, L, F32)
    ids = torch.arange(T, device="cuda", dtype=I32) % L
    plan = qm.lora_plan(ids, L)
    want = qm.lora_add(base, x, a, b, plan, scales=s)
    b[0, 77, 3] = float("inf")
    base[T - 1, 9] = -float("inf")
    got = qm.lora_add(base, x, a, b, plan, scales=s)
    bad = torch.zeros((T, N), dtype=torch.bool, device="cuda")
    bad[ids == 0, 77] = True
    assert not torch.isfinite(got[bad]).any() and got[T - 1, 9] == -float("inf")
    bad[T - 1, 9] = True
    assert torch.equal(got[~bad], want[~bad])


# ---------------------------------------------------- offsets past 32 bits

def far_rows(T, n, step, dtype):
    """T rows of n values, step apart: only what is used is ever touched."""
    buf = torch.empty((T - 1) * step + n, dtype=dtype, device="cuda")
    return buf.as_strided((T, n), (step, 1))


@pytest.mark.parametrize("T", [3, 9])
def test_lora_of_rows_far_apart(T):
    K, N, r, L = 64, 96, 16, 2
    g = gen(T)
    x, a, b, base, s = B.lora_case(g, T, K, N, r, L, BF16)
    ids = torch.arange(T, device="cuda", dtype=I32) % L
    step = 2 ** 32 // (T - 1) + 64
    fx, fb, fo = far_rows(T, K, step, BF16), far_rows(T, N, step, BF16), far_rows(T, N, step + 8, BF16)
    fx.copy_(x)
    fb.copy_(base)
    plan = qm.lora_plan(ids, L)
    qm.lora_add(fb, fx, a, b, plan, scales=s, out=fo)
    assert torch.equal(fo, qm.lora_add(base, x, a, b, plan, scales=s))


@pytest.mark.parametrize("T", [2, 6])
def test_lora_of_large_adapters(T):
    """a and b of more than 2^32 values, of which the last adapter is used."""
    K, N, r, L = 16384, 20000, 256, 1024
    g = gen(T)
    x, a1, b1, base, s = B.lora_case(g, T, K, N, r, 1, F32)
    a = torch.empty((L, r, K), dtype=BF16, device="cuda")
    b = torch.empty((L, N, r), dtype=BF16, device="cuda")
    a[L - 1], b[L - 1] = a1[0], b1[0]
    ids = torch.full((T,), L - 1, dtype=I32, device="cuda")
    got = qm.lora_add(base, x, a, b, qm.lora_plan(ids, L))
    want, bound = B.lora(base, x, a1, b1, torch.zeros_like(ids))
    B.check_rounded(got, want, bound, F32)


@pytest.mark.parametrize("V", [700, 50001])
def test_scores_of_rows_far_apart(V):
    T = 5
    l = (2.5 * torch.randn((T, V), generator=gen(V), device="cuda")).to(BF16)
    far = far_rows(T, V, 2 ** 30 + 5, BF16)
    far.copy_(l)
    tok = torch.randint(0, V, (T, 3), generator=gen(1), device="cuda", dtype=I32)
    B.check_scores(l, tok, 9, qm.token_logprobs(far, tok, top=9, entropy=True))


def test_rows_behind_the_last_stay():
    """Through the C entry points, with room behind every output."""
    T, L, K, N, r, V, top = 37, 5, 64, 72, 8, 3001, 4
    g = gen(3)
    x, a, b, base, s = B.lora_case(g, T, K, N, r, L, BF16)
    ids = torch.randint(0, L, (T,), generator=g, device="cuda", dtype=I32)
    lb, st = qm.lib(), torch.cuda.current_stream().cuda_stream
    n = lb.moe_lora_items(T, L)
    off, perm, items = (torch.full((k,), 77, dtype=I32, device="cuda") for k in (L + 2 + 8, T + 8, 4 * n + 8))
    assert lb.moe_lora_plan(T, L, ids.data_ptr(), off.data_ptr(), perm.data_ptr(), items.data_ptr(), None, 0, st) == 0
    assert (off[L + 2:] == 77).all() and (perm[T:] == 77).all() and (items[4 * n:] == 77).all()
    out = torch.full((T + 3, N), 77.0, dtype=BF16, device="cuda")
    wn = lb.moe_lora_add_workspace_bytes(T, K, N, r, L)
    ws = torch.full((wn + 64,), 77, dtype=torch.uint8, device="cuda")
    assert lb.moe_lora_add(T, K, N, r, L, x.data_ptr(), K, a.data_ptr(), b.data_ptr(), s.data_ptr(), perm.data_ptr(), items.data_ptr(),
                           base.data_ptr(), N, out.data_ptr(), N, qm.MOE_TYPE_BF16, ws.data_ptr(), wn, st) == 0
    assert (out[T:] == 77).all() and (ws[wn:] == 77).all()
    assert torch.equal(out[:T], qm.lora_add(base, x, a, b, qm.lora_plan(ids, L), scales=s))
    l = torch.randn((T, V), generator=g, device="cuda")
    tok = torch.randint(0, V, (T, 2), generator=g, device="cuda", dtype=I32)
    lp, ent, tlp = (torch.full((k,), 77.0, device="cuda") for k in (2 * T + 8, T + 8, top * T + 8))
    top_ids = torch.full((top * T + 8,), 77, dtype=I32, device="cuda")
    wn = lb.moe_token_logprobs_workspace_bytes(T, V, top)
    ws = torch.full((wn + 64,), 77, dtype=torch.uint8, device="cuda")
    assert lb.moe_token_logprobs(T, V, l.data_ptr(), qm.MOE_TYPE_F32, V, tok.data_ptr(), 2, lp.data_ptr(), ent.data_ptr(), top,
                                 top_ids.data_ptr(), tlp.data_ptr(), ws.data_ptr() if wn else None, wn, st) == 0
    for t, k in ((lp, 2 * T), (ent, T), (tlp, top * T), (top_ids, top * T)):
        assert (t[k:] == 77).all()
    assert (ws[wn:] == 77).all()
    B.check_scores(l, tok, top, (lp[:2 * T].view(T, 2), ent[:T], top_ids[:top * T].view(T, top), tlp[:top * T].view(T, top)))
