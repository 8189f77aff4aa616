"""The operators of a batch of many requests on the GPU against float64
(tests/batch_ref.py), at the sizes, ids, masks and layouts where a run, a part
or a list can go wrong."""

import math

import pytest
import torch

import batch_ref as B
import quantized_routed_moe_amd as qm
from batch_ref import gen

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


# ------------------------------------------------------------------- plan

def some_ids(g, T, L, kind):
    if kind == "one":
        return torch.full((T,), L - 1, dtype=I32, device="cuda")
    if kind == "none":
        return torch.full((T,), -1, dtype=I32, device="cuda")
    if kind == "wild":              # ids on both sides of the range, the largest and smallest ints among them
        ids = torch.randint(-2, L + 2, (T,), generator=g, device="cuda", dtype=I32)
        ids[::7], ids[3::11] = 2 ** 31 - 1, -2 ** 31
        return ids
    if kind == "runs":
        return torch.randint(0, L, (T // 40 + 1,), generator=g, device="cuda", dtype=I32).repeat_interleave(40)[:T].contiguous()
    return torch.randint(0, L, (T,), generator=g, device="cuda", dtype=I32)


@pytest.mark.parametrize("kind", ["random", "one", "none", "wild", "runs"])
@pytest.mark.parametrize("T,L", [(1, 1), (1, 1024), (2, 3), (63, 7), (64, 64), (65, 1), (200, 31), (256, 1024), (257, 32), (1000, 127),
                                 (4097, 128), (8192, 1024), (8192, 5), (8193, 1024), (20000, 33), (200000, 1000)])
def test_plan(T, L, kind):
    ids = some_ids(gen(T + L), T, L, kind)
    given = ids.clone()
    B.check_plan(qm.lora_plan(ids, L), ids, L)
    assert torch.equal(ids, given)


def test_plan_of_no_tokens():
    p = qm.lora_plan(torch.empty(0, dtype=I32, device="cuda"), 5)
    assert p.perm.numel() == 0 and p.items.shape == (0, 4) and (p.offsets == 0).all()


def test_plan_refusals():
    ids = torch.zeros(10, dtype=I32, device="cuda")
    for bad in (lambda: qm.lora_plan(ids, 0), lambda: qm.lora_plan(ids, -4), lambda: qm.lora_plan(ids, 1025)):
        with pytest.raises(qm.MoeError) as e:
            bad()
        assert e.value.code == qm.MOE_ERR_SHAPE
    for bad in (ids.long(), ids[::2]):
        with pytest.raises(ValueError):
            qm.lora_plan(bad, 3)


# --------------------------------------------------------------- adapters

def check_lora(T, K, N, r, L, dtype, ids, seed=0, scaled=True):
    g = gen(seed + T + K + N + r)
    x, a, b, base, s = B.lora_case(g, T, K, N, r, L, dtype)
    s = s if scaled else None
    plan = qm.lora_plan(ids, L)
    before = base.clone()
    got = qm.lora_add(base, x, a, b, plan, scales=s)
    assert torch.equal(base, before)
    want, bound = B.lora(base, x, a, b, ids, s)
    B.check_rounded(got, want, bound, dtype, f"T={T} K={K} N={N} r={r} L={L}")
    none = (ids < 0) | (ids >= L)
    assert torch.equal(got[none], base[none])
    # in place: the same bits
    again = base.clone()
    assert qm.lora_add(again, x, a, b, plan, scales=s, out=again) is again
    assert torch.equal(again, got)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("K,N,r", [(32, 1, 8), (64, 15, 16), (96, 64, 24), (1056, 130, 40), (160, 1111, 64), (4096, 257, 72),
                                   (2048, 512, 128), (32, 300, 256), (4128, 33, 8)])
@pytest.mark.parametrize("T,L", [(1, 1), (2, 5), (17, 1), (33, 4), (65, 3), (200, 64), (700, 9)])
def test_lora(T, L, K, N, r, dtype):
    ids = some_ids(gen(T + L), T, L, "wild" if T > 2 else "random")
    check_lora(T, K, N, r, L, dtype, ids, scaled=r != 24)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [1, 5, 64, 300, 2048])
def test_lora_long(T, dtype):
    check_lora(T, 4096, 4096, 16, 16, dtype, some_ids(gen(T), T, 16, "runs" if T > 100 else "random"))


@pytest.mark.parametrize("kind", ["one", "none", "runs"])
def test_lora_ids(kind):
    check_lora(130, 512, 200, 16, 6, BF16, some_ids(gen(2), 130, 6, kind))


def test_lora_many_adapters():
    """As many adapters as a call takes, most of them without a token."""
    ids = torch.tensor([1023, 0, 511, 511, -1, 1024, 1000], dtype=I32, device="cuda")
    check_lora(7, 256, 96, 8, 1024, F32, ids)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_lora_strided(dtype):
    """Rows apart, at strides that allow whole 16 bytes and at one that does
    not; what lies between the rows stays as it was; one row of x, and of base,
    for all."""
    T, K, N, r, L = 40, 128, 200, 16, 3
    g = gen(9)
    x, a, b, base, s = B.lora_case(g, T, K, N, r, L, dtype)
    ids = some_ids(g, T, L, "random")
    plan = qm.lora_plan(ids, L)
    want = qm.lora_add(base, x, a, b, plan, scales=s)
    bx = torch.full((T, K + 24), 9.0, dtype=BF16, device="cuda")
    bx[:, 8:8 + K] = x
    for pad in (8, 7):
        bb = torch.full((T, N + pad), 7.0, dtype=dtype, device="cuda")
        bb[:, :N] = base
        bo = torch.full((T, N + 2 * pad), 5.0, dtype=dtype, device="cuda")
        assert torch.equal(qm.lora_add(bb[:, :N], bx[:, 8:8 + K], a, b, plan, scales=s, out=bo[:, :N]), want)
        assert (bo[:, N:] == 5).all()
        qm.lora_add(bb[:, :N], x, a, b, plan, scales=s, out=bb[:, :N])
        assert torch.equal(bb[:, :N], want) and (bb[:, N:] == 7).all()
    one = qm.lora_add(base[:1].expand(T, N), x[:1].expand(T, K), a, b, plan, scales=s)
    assert torch.equal(one, qm.lora_add(base[:1].repeat(T, 1), x[:1].repeat(T, 1), a, b, plan, scales=s))


def test_lora_non_finite_values_stay_in_their_rows():
    """A NaN in one token's row, an infinity in one adapter: the other tokens'
    rows are what they are without."""
    T, K, N, r, L = 50, 256, 100, 16, 4
    g = gen(4)
    x, a, b, base, s = B.lora_case(g, T, K, N, r, L, F32)
    ids = some_ids(g, T, L, "random")
    plan = qm.lora_plan(ids, L)
    want = qm.lora_add(base, x, a, b, plan, scales=s)
    x[7, 100] = float("nan")
    a[2, 5, 33] = float("inf")
    base[9, 4] = float("nan")
    got = qm.lora_add(base, x, a, b, plan, scales=s)
    bad = (ids == 2)
    bad[7] = True
    assert not torch.isfinite(got[bad]).any()
    keep = ~bad
    want[9, 4] = float("nan")
    assert torch.equal(got[keep].nan_to_num(nan=3e38), want[keep].nan_to_num(nan=3e38))


def test_lora_rows_do_not_depend_on_the_batch():
    """A token's result is the same bits alone, among others and at another
    place in the batch, while the parts of K are the same."""
    T, K, N, r, L = 12, 512, 320, 16, 3
    g = gen(6)
    x, a, b, base, s = B.lora_case(g, T, K, N, r, L, F32)
    ids = some_ids(g, T, L, "random")
    all_ = qm.lora_add(base, x, a, b, qm.lora_plan(ids, L), scales=s)
    back = torch.arange(T - 1, -1, -1, device="cuda")
    turned = qm.lora_add(base[back], x[back], a, b, qm.lora_plan(ids[back].contiguous(), L), scales=s)
    assert torch.equal(turned[back], all_)


def test_lora_follows_no_entry_out_of_range():
    """A plan overwritten with entries outside their ranges: nothing is
    followed, what is sound is done, nothing behind the result is written."""
    T, K, N, r, L = 70, 64, 80, 8, 4
    g = gen(8)
    x, a, b, base, s = B.lora_case(g, T, K, N, r, L, F32)
    ids = torch.zeros(T, dtype=I32, device="cuda")
    ids[64:] = 2
    plan = qm.lora_plan(ids, L)
    want = qm.lora_add(base, x, a, b, plan, scales=s)
    perm = plan.perm.clone()
    perm[3], perm[5], perm[66] = -1, T, 2 ** 31 - 1
    items = plan.items.clone()
    items[2] = torch.tensor([7, 0, 5, 0])              # no such adapter
    items[3] = torch.tensor([1, -9, -4, 0])
    buf = torch.full((T + 8, N), 3.0, device="cuda")
    out = buf[:T]
    qm.lora_add(base, x, a, b, qm.LoraPlan(T, L, perm, plan.offsets, items), scales=s, out=out)
    skipped = torch.zeros(T, dtype=torch.bool, device="cuda")
    skipped[[3, 5, 66]] = True
    assert torch.equal(out[~skipped], want[~skipped]) and (out[skipped] == 3).all() and (buf[T:] == 3).all()


def test_lora_refusals():
    g = gen(1)
    x, a, b, base, s = B.lora_case(g, 6, 64, 40, 8, 3, BF16)
    plan = qm.lora_plan(torch.zeros(6, dtype=I32, device="cuda"), 3)
    ok = dict(base=base, x=x, a=a, b=b, plan=plan, scales=s)
    qm.lora_add(**ok)
    other = qm.lora_plan(torch.zeros(5, dtype=I32, device="cuda"), 3)
    for bad in (dict(x=x.float()), dict(x=x[:5]), dict(a=a.float()), dict(b=b[:, :, :4]), dict(b=b[:2]), dict(scales=s.double()),
                dict(scales=s[:2]), dict(plan=other), dict(plan=qm.lora_plan(torch.zeros(6, dtype=I32, device="cuda"), 2)),
                dict(base=base.half()), dict(base=base.t()), dict(out=base.float()), dict(out=base[:5]), dict(x=x.cpu()),
                dict(a=a.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            qm.lora_add(**{**ok, **bad})
    wide = torch.zeros((6, 96), dtype=BF16, device="cuda")
    for bad, code in ((dict(x=wide[:, 4:68]), qm.MOE_ERR_ALIGN), (dict(base=wide[:, 1:41]), qm.MOE_ERR_ALIGN),
                      (dict(base=wide[:1, :40].expand(6, 40), out=wide[:, :40]), qm.MOE_ERR_UNSUPPORTED)):
        with pytest.raises(qm.MoeError) as e:
            qm.lora_add(**{**ok, **bad})
        assert e.value.code == code


# ----------------------------------------------------------------- scores

def logits_of(g, T, V, dtype, spread=2.5):
    l = torch.randn((T, V), generator=g, device="cuda") * spread
    for i in range(3):
        l.scatter_(1, torch.randint(0, V, (T, 1), generator=g, device="cuda"), 9.0 + 2 * i)
    return l.to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("top", [0, 1, 5, 20, 64])
@pytest.mark.parametrize("T,V", [(1, 1), (3, 2), (5, 7), (2, 8), (4, 15), (3, 17), (7, 64), (2, 65), (9, 100), (3, 511), (70, 1000), (2, 2049),
                                 (1, 8192), (3, 8193), (1, 50001), (600, 333), (3, 128256), (520, 5003)])
def test_scores(T, V, top, dtype):
    g = gen(T + V + top)
    l = logits_of(g, T, V, dtype)
    top = min(top, V)
    given = (top % 3) + 1
    tok = torch.randint(0, V, (T, given), generator=g, device="cuda", dtype=I32)
    before = l.clone()
    got = qm.token_logprobs(l, tok, top=top, entropy=top != 1)
    assert torch.equal(l, before)
    B.check_scores(l, tok, top, got, f"T={T} V={V}")


def test_scores_outputs_alone():
    g = gen(3)
    l = logits_of(g, 20, 3001, BF16)
    tok = torch.randint(0, 3001, (20,), generator=g, device="cuda", dtype=I32)
    lp, ent, ids, tlp = qm.token_logprobs(l, tok, top=4, entropy=True)
    assert lp.shape == (20,) and ids.dtype == I32
    a = qm.token_logprobs(l, tok)
    assert torch.equal(a[0], lp) and a[1:] == (None, None, None)
    b = qm.token_logprobs(l, entropy=True)
    assert torch.equal(b[1], ent) and b[0] is None and b[2] is None
    c = qm.token_logprobs(l, top=4)
    assert torch.equal(c[2], ids) and torch.equal(c[3], tlp)
    many = qm.token_logprobs(l, tok[:, None].expand(20, 200).contiguous())
    assert torch.equal(many[0], lp[:, None].expand(20, 200))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V,pad", [(100, 1), (1000, 3), (4097, 0), (50001, 5)])
def test_scores_strided(V, pad, dtype):
    """Rows that start at any value, with what lies between them larger than
    all of theirs."""
    T = 9
    buf = torch.full((T, V + pad), 1e6, device="cuda").to(dtype)
    l = logits_of(gen(V), T, V, dtype)
    buf[:, :V] = l
    tok = torch.randint(0, V, (T,), generator=gen(1), device="cuda", dtype=I32)
    B.check_scores(l, tok, 10, qm.token_logprobs(buf[:, :V], tok, top=10, entropy=True))
    one = qm.token_logprobs(l[:1], tok[:1], top=10, entropy=True)
    B.check_scores(l[:1], tok[:1], 10, one)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,V", [(2, 300), (3, 20000), (600, 2500), (1, 128256)])
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "two", "lowest", "highest", "offset", "zeros"])
def test_scores_of_orders_and_extremes(kind, T, V, dtype):
    """Ties go to the lowest place wherever they lie; orders that fill the
    lists again and again; the type's lowest value as a mask; logits far from 0."""
    big = torch.finfo(dtype).max
    i = torch.arange(V, device="cuda", dtype=F32)
    if kind == "equal":
        row = torch.full((V,), 3.0, device="cuda")
    elif kind == "rising":
        row = i * (20.0 / V)
    elif kind == "falling":
        row = -i * (20.0 / V)
    elif kind == "two":
        row = torch.where(i % 37 == 5, 2.0, -1.0)
    elif kind == "lowest":          # all but a few masked by the lowest finite value
        row = torch.where((i % 1000 == 7) | (i == V - 1), i % 5, -big)
    elif kind == "highest":
        row = torch.where(i == V // 2, big, 1.0)
    elif kind == "offset":
        row = 1000.0 + 8 * torch.sin(i)
    else:                           # zeros of both signs are equal
        row = torch.where(i % 2 == 0, -0.0, 0.0)
    l = row.to(dtype).expand(T, V).contiguous()
    l[T - 1] = l[T - 1].roll(3)
    tok = torch.randint(0, V, (T, 2), generator=gen(V), device="cuda", dtype=I32)
    top = 30
    B.check_scores(l, tok, top, qm.token_logprobs(l, tok, top=top, entropy=True), kind)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,V", [(6, 200), (7, 20000), (520, 2304)])
def test_scores_of_masked_rows(T, V, dtype):
    """-inf: a part of the row, all but one place, all but fewer than `top`,
    everything; what is left counts and the lowest masked places follow."""
    l = logits_of(gen(V), T, V, dtype)
    l[0, ::2] = -math.inf
    l[1] = -math.inf
    l[1, V - 3] = 2.0
    l[2] = -math.inf
    l[3, :] = -math.inf
    l[3, [0, 1, 5, 70, 150, V - 1]] = torch.tensor([1.0, 4.0, 4.0, -7.0, 0.0, 2.0], device="cuda").to(dtype)
    l[4, 17:] = -math.inf
    tok = torch.randint(0, V, (T, 3), generator=gen(V), device="cuda", dtype=I32)
    tok[1, 0] = V - 3
    B.check_scores(l, tok, 64, qm.token_logprobs(l, tok, top=64, entropy=True))
    lp, ent, ids, tlp = qm.token_logprobs(l[1:3].contiguous(), tok[1:3].contiguous(), top=3, entropy=True)
    assert lp[0, 0] == 0 and (ent == 0).all() and ids.tolist() == [[V - 3, 0, 1], [0, 1, 2]]
    assert tlp[0].tolist() == [0.0, -math.inf, -math.inf] and (lp[1] == -math.inf).all() and (tlp[1] == -math.inf).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,V", [(5, 200), (4, 20000), (530, 2304)])
def test_scores_of_nan_and_infinite_logits(T, V, dtype):
    """Rows with a NaN or +inf give NaN and -1; their neighbours are not
    touched, and a token outside the row is not followed."""
    l = logits_of(gen(V), T, V, dtype)
    tok = torch.randint(0, V, (T, 4), generator=gen(V), device="cuda", dtype=I32)
    want = qm.token_logprobs(l, tok, top=7, entropy=True)
    l[0, V - 1] = math.nan
    l[2, 0] = math.inf
    l[3, V // 2:] = math.nan
    l[3, :V // 2] = -math.inf
    bad = [0, 2, 3]
    tok2 = tok.clone()
    tok2[1, 0], tok2[1, 1], tok2[1, 2] = -1, V, 2 ** 31 - 1
    lp, ent, ids, tlp = qm.token_logprobs(l, tok2, top=7, entropy=True)
    assert torch.isnan(lp[bad]).all() and torch.isnan(ent[bad]).all() and torch.isnan(tlp[bad]).all() and (ids[bad] == -1).all()
    assert torch.isnan(lp[1, :3]).all() and lp[1, 3] == want[0][1, 3]
    keep = [t for t in range(T) if t not in bad]
    for got, w in zip((ent, ids, tlp), want[1:]):
        assert torch.equal(got[keep], w[keep])
    assert torch.equal(lp[keep[1:]], want[0][keep[1:]])


def test_scores_refusals():
    l = torch.zeros((4, 100), device="cuda")
    tok = torch.zeros(4, dtype=I32, device="cuda")
    for bad in (dict(logits=l.half()), dict(logits=l[0]), dict(logits=l.t()), dict(tokens=tok.long()), dict(tokens=tok[:3]),
                dict(tokens=tok.cpu()), dict(tokens=tok.view(4, 1, 1))):
        with pytest.raises(ValueError):
            qm.token_logprobs(**{**dict(logits=l, tokens=tok), **bad})
    for bad, code in ((dict(top=65), qm.MOE_ERR_SHAPE), (dict(logits=l[:, :3], top=4), qm.MOE_ERR_SHAPE),
                      (dict(tokens=None), qm.MOE_ERR_NULL), (dict(logits=l[:, 1:]), qm.MOE_ERR_ALIGN),
                      (dict(logits=torch.zeros((1, 100000), device="cuda"), tokens=tok[:1],
                            ws=torch.empty(16, dtype=torch.uint8, device="cuda")), qm.MOE_ERR_WORKSPACE)):
        with pytest.raises(qm.MoeError) as e:
            qm.token_logprobs(**{**dict(logits=l, tokens=tok), **bad})
        assert e.value.code == code


def test_empty_batches():
    e = lambda *s, dt=BF16: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    plan = qm.lora_plan(e(0, dt=I32), 2)
    out = qm.lora_add(e(0, 40), e(0, 64), torch.zeros((2, 8, 64), dtype=BF16, device="cuda"),
                      torch.zeros((2, 40, 8), dtype=BF16, device="cuda"), plan)
    assert out.shape == (0, 40)
    lp, ent, ids, tlp = qm.token_logprobs(e(0, 50), e(0, dt=I32), top=3, entropy=True)
    assert lp.shape == (0,) and ent.shape == (0,) and ids.shape == tlp.shape == (0, 3)
