"""The definitions of the operators of a batch of many requests in float64
(torch, on whatever device the inputs are), the inputs of their tests, and
error bounds by counting roundings.  U32 is half a step of fp32 relative to the
value, and so on."""

import math

import torch

U32, UBF16 = 2.0 ** -24, 2.0 ** -8


def gen(seed, dev="cuda"):
    return torch.Generator(device=dev).manual_seed(seed)


def check_rounded(got, want, bound, dtype, what=""):
    """got is within `bound` and one rounding to its type of `want`."""
    u = {torch.float32: U32, torch.bfloat16: UBF16}[dtype]
    assert got.dtype == dtype and got.shape == want.shape, what
    assert torch.isfinite(got.double()).all(), f"{what}: non-finite"
    over = (got.double() - want).abs() - bound - u * (want.abs() + bound)
    assert (over <= 0).all(), f"{what}: over the bound by {float(over.max()):.3e}"


# ------------------------------------------------------------------ adapters

def groups(ids, L):
    return torch.where((ids >= 0) & (ids < L), ids, L).long()


def check_plan(plan, ids, L):
    """perm and offsets are those of a stable sort by group, and the items its
    runs of at most 64, in order."""
    g = groups(ids, L)
    T = ids.numel()
    counts = torch.bincount(g, minlength=L + 1)
    off = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    assert torch.equal(plan.offsets.long(), off)
    assert torch.equal(plan.perm.long(), torch.sort(g, stable=True).indices)
    want = [(e, r, min(r + 64, b), 0) for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:])) for r in range(a, b, 64)]
    items = plan.items.tolist()
    assert len(want) <= len(items) <= T // 64 + min(L + 1, T) + 1
    assert [tuple(i) for i in items[:len(want)]] == want
    assert all(i == [-1, 0, 0, 0] for i in items[len(want):])


def lora(base, x, a, b, ids, scales=None):
    """(out, bound) of a token's adapter, g its id:

    v: a wave adds at most ceil(ceil(K/128)/4) steps of 128 exact products, then
    4 waves and at most 8 parts of K are added (few tokens: a lane adds at most
    ceil(ceil(K/128)/8) steps of 4 pairs, off by 2^1.5 halves each, then 34
    partial sums, which is less); v in three bf16 parts holds it to half a step;
    3 r products and one more rounding each for the sum of parts' magnitudes,
    the factor and the addition to base."""
    out, bound = base.double().clone(), torch.zeros_like(base, dtype=torch.float64)
    K, r = a.shape[2], a.shape[1]
    deep = -(-(-(-K // 128)) // 4) * 128 + 16
    for e in torch.unique(ids).tolist():
        if not 0 <= e < a.shape[0]:
            continue
        t = torch.nonzero(ids == e)[:, 0]
        xd, ad, bd = x[t].double(), a[e].double().t().contiguous(), b[e].double().t().contiguous()
        s = 1.0 if scales is None else float(scales[e])
        v = xd @ ad
        dv = deep * U32 * (xd.abs() @ ad.abs())
        d = v @ bd
        dd = (dv + U32 * v.abs()) @ bd.abs() + (3 * r + 3) * U32 * ((v.abs() + dv) @ bd.abs())
        out[t] += s * d
        bound[t] = abs(s) * dd + U32 * (base[t].double().abs() + abs(s) * (d.abs() + dd))
    return out, bound


def lora_case(g, T, K, N, r, L, dtype, dev="cuda"):
    """x, a, b, base, scales: results of order one."""
    x = torch.randn((T, K), generator=g, device=dev).to(torch.bfloat16)
    a = (torch.randn((L, r, K), generator=g, device=dev) / math.sqrt(K)).to(torch.bfloat16)
    b = (torch.randn((L, N, r), generator=g, device=dev) / math.sqrt(r)).to(torch.bfloat16)
    base = torch.randn((T, N), generator=g, device=dev).to(dtype)
    return x, a, b, base, torch.exp2(2 * torch.rand(L, generator=g, device=dev) - 1)


# ------------------------------------------------------------------ scores

def scores(logits):
    """Per row in float64: log p [T][V], entropy, and (bounds) of each.

    S: every term is off by 2|d| + 3 halves (l - m, the product with log2 e, the
    exponential), each lane adds at most V / 64 + 8 of them (one wave has a
    whole row when it is short), a raise of the maximum costs 4 on what is
    there, at most one for each of V / 256 rounds and 64 joins.  ln S: a step of
    its value and the relative error of S; d and the difference: half a step.  U
    likewise, its terms weighted by |d|."""
    l = logits.double()
    V = l.shape[1]
    m = l.amax(1, keepdim=True)
    empty = torch.isinf(m) & (m < 0)
    d = torch.where(empty, -math.inf, l - torch.where(empty, 0.0, m))
    e = torch.exp(d)
    S = e.sum(1, keepdim=True)
    lnS = torch.where(empty, 0.0, torch.log(torch.where(empty, 1.0, S)))
    fin = torch.where(e > 0, d, 0.0)
    p = e / torch.where(empty, 1.0, S)
    n = V / 64 + 8 + 4 * (V / 256 + 64)
    dS = U32 * ((p * (2 * fin.abs() + 3)).sum(1, keepdim=True) + n)
    lp = d - lnS
    far = torch.where(torch.isinf(d), 0.0, d)
    dlp = dS + U32 * (2 * lnS.abs() + far.abs() + (far - lnS).abs())
    U = (p * fin).sum(1, keepdim=True)
    H = (lnS - U)[:, 0]
    dU = U32 * (p * fin.abs() * (2 * fin.abs() + 5 + n)).sum(1, keepdim=True) + U.abs() * dS
    dH = (dS + dU + U32 * (2 * lnS.abs() + 2 * U.abs() + H[:, None].abs()))[:, 0]
    return lp, dlp, H, dH


def check_close(got, want, bound, what=""):
    """Within the bound where want is finite, equal where it is not."""
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf), f"{what}: infinities"
    assert (got[inf] < 0).all(), what
    over = ((got.double() - want).abs() - bound)[~inf]
    assert not torch.isnan(got).any(), f"{what}: NaN"
    assert over.numel() == 0 or float(over.max()) <= 0, f"{what}: over the bound by {float(over.max()):.3e}"


def check_scores(logits, tokens, top, got, what=""):
    """All outputs of token_logprobs against the definitions, in parts of rows."""
    logprobs, entropy, ids, top_lp = got
    for t in range(0, logits.shape[0], 256):
        r = slice(t, t + 256)
        lp, dlp, H, dH = scores(logits[r])
        if tokens is not None:
            tok = tokens[r].long().view(lp.shape[0], -1)
            check_close(logprobs[r].view(tok.shape), lp.gather(1, tok), dlp.gather(1, tok), f"{what} logprobs")
        if entropy is not None:
            check_close(entropy[r], H, dH, f"{what} entropy")
        if top:
            order = torch.sort(logits[r].double() + 0.0, dim=1, descending=True, stable=True).indices[:, :top]
            assert torch.equal(ids[r].long(), order), f"{what} top_ids"
            check_close(top_lp[r], lp.gather(1, order), dlp.gather(1, order), f"{what} top_logprobs")
