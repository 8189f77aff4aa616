"""Inputs of the operators of a batch of many requests whose results are known to
the bit, or to the rounding of one logarithm: what a bound that counts the worst
roundings of long sums would let through shows there (torch, on whatever device
the generator is)."""

import math

import torch

U32 = 2.0 ** -24


# ------------------------------------------------------------------ adapters

def lora_case(g, T, K, N, r, L, ids):
    """(base, x, a, b, scales, out): v of every token and rank is a number of its own with
    24 bits, the sum of three bf16 numbers of 8 bits each at three places of K that are
    the rank's, where a is 1; x is anything elsewhere, where a is 0.  All partial sums of the
    three have 24 bits too, so v is exact in whatever order it is added.  A column
    takes one rank, times a power of two, and so does the factor: out is exact in fp32."""
    dev = ids.device
    assert 3 * r <= K
    m = torch.randint(2 ** 23, 2 ** 24, (T, r), generator=g, device=dev)
    m |= 1                                                      # the last bit too
    sign = 1 - 2 * torch.randint(0, 2, (T, r), generator=g, device=dev)
    parts = torch.stack([m >> 16 << 16, m & 0xff00, m & 0xff], 2) * sign[:, :, None]       # [T][r][3]
    places = torch.stack([torch.randperm(K, generator=g, device=dev)[:3 * r].view(r, 3) for _ in range(L)])
    x = torch.randn((T, K), generator=g, device=dev)
    who = ids.long()
    has = (who >= 0) & (who < L)
    who = torch.where(has, who, 0)
    x.scatter_(1, places[who].view(T, 3 * r), (parts.double() * 2.0 ** -23).float().view(T, 3 * r))
    a = torch.zeros((L, r, K), device=dev).scatter_(2, places, 1.0)
    rank = torch.stack([torch.randperm(N, generator=g, device=dev) % r for _ in range(L)])    # of each column
    b = torch.zeros((L, N, r), device=dev)
    times = torch.exp2(torch.randint(-3, 4, (L, N), generator=g, device=dev).float())
    b.scatter_(2, rank[:, :, None], times[:, :, None])
    scales = torch.exp2(torch.randint(-3, 4, (L,), generator=g, device=dev).float())
    v = m.double() * 2.0 ** -23 * sign
    out = torch.where(has[:, None], v.gather(1, rank[who]) * times[who].double() * scales[who].double()[:, None], 0.0)
    base = torch.zeros((T, N), device=dev)
    assert torch.equal(out.float().double(), out)
    return base, x.to(torch.bfloat16), a.to(torch.bfloat16), b.to(torch.bfloat16), scales, out.float()


def in_parts(v, n):
    """The sum of the first n of a float's bf16 parts, each the nearest to what is left."""
    s = torch.zeros_like(v)
    for _ in range(n):
        s = s + (v - s).to(torch.bfloat16).float()
    return s


def sum_bound(K, waves):
    """Of the mean square of v's error against that of v, for products of random sign:
    each of `waves` waves adds K / waves of them, at most one by one, and the roundings
    of partial sums, half a step of each at most, are independent of each other; the mean
    square of the i-th partial sum is i times that of a product, so that of a wave's error is
    U32^2 n^2 / 2 of them and that of all n waves / (n waves) = n / 2 of v's.  waves + 8 further
    sums (waves, parts, places of a wave, the product with b) add as many squares."""
    n = K / waves
    return U32 ** 2 * (n / 2 + waves + 8)


# -------------------------------------------------------------------- scores

LOW = 200.0            # e^-200 is 0 in fp32, and its logit finite


def counted(g, T, V, dtype, kind, per):
    """(here [T][V], logits): every row holds one value at the places `here` and nothing
    that counts elsewhere: -inf in even rows, a far lower value in odd ones.  So the sum of
    exponentials is the count of those places, exactly, and each logarithm ln of a whole
    number, which a single value too many or too few changes."""
    dev = g.device
    i = torch.arange(V, device=dev)
    if kind == "all":
        here = torch.ones((T, V), dtype=torch.bool, device=dev)
    elif kind == "half":
        here = torch.rand((T, V), generator=g, device=dev) < 0.5
    elif kind == "few":
        here = torch.zeros((T, V), dtype=torch.bool, device=dev)
        here.scatter_(1, torch.randint(0, V, (T, 9), generator=g, device=dev), True)
    elif kind == "ends":               # what lies outside whole 16 bytes, and a chunk beside it
        here = ((i < 2 * per) | (i >= V - 2 * per)).expand(T, V).clone()
    else:                              # first and last chunks of a wave's 64, wherever the row begins
        at = torch.arange(T, device=dev)[:, None] % per + i
        chunk = at // per % 64
        here = (chunk == 0) | (chunk == 63)
    here[torch.arange(T, device=dev), torch.randint(0, V, (T,), generator=g, device=dev)] = True
    far = torch.where(torch.arange(T, device=dev) % 2 == 0, -math.inf, 3.0 - LOW)[:, None]
    return here, torch.where(here, 3.0, far).to(dtype)


def check_counted(here, logits, tokens, top, got, what=""):
    """ln of a count: a step of its value (the logarithm) and half a step (the
    difference); of a far value also half a step of each difference."""
    logprobs, entropy, ids, top_lp = got
    T, V = here.shape
    ln = torch.log(here.sum(1).double())[:, None]
    far = torch.where(torch.arange(T, device=here.device) % 2 == 0, -math.inf, -LOW).double()[:, None]
    want = torch.where(here, 0.0, far) - ln
    bound = U32 * (3 * ln + torch.where(here | torch.isinf(far), 0.0, 2 * (LOW + ln)))

    def close(g, w, b, name):
        inf = torch.isinf(w)
        assert torch.equal(torch.isinf(g), inf) and (g[inf] < 0).all() and not torch.isnan(g).any(), f"{what} {name}"
        over = ((g.double() - w).abs() - b)[~inf]
        assert over.numel() == 0 or float(over.max()) <= 0, f"{what} {name}: over the bound by {float(over.max()):.3e}"

    if tokens is not None:
        tok = tokens.long()
        close(logprobs, want.gather(1, tok), bound.gather(1, tok), "logprobs")
    if entropy is not None:
        close(entropy, ln[:, 0], 3 * U32 * ln[:, 0], "entropy")
    if top:
        order = torch.sort(~here, dim=1, stable=True).indices[:, :top]
        assert torch.equal(ids.long(), order), f"{what} top_ids"
        close(top_lp, want.gather(1, order), bound.gather(1, order), "top_logprobs")


def scores_mean_square(logits):
    """(log p, H, bounds of the mean squares of their errors over the rows) in float64, as
    batch_ref.scores but for roundings that are independent of each other, so that their
    squares add: of a term's share of S three halves and two |d| halves; of a lane's sums,
    at most V / 64 + 8, half a step of S each at most; of raises, 4 halves of S each, V / 256
    + 64 of them at most.  What the exponential may be off in one direction, a step, is
    added to the root."""
    l = logits.double()
    V = l.shape[1]
    d = l - l.amax(1, keepdim=True)
    e = torch.exp(d)
    S = e.sum(1, keepdim=True)
    ln, p = torch.log(S), e / S
    U = (p * d).sum(1, keepdim=True)
    n = V / 64 + 8 + 16 * (V / 256 + 64)
    rel = torch.sqrt((p * (2 * d.abs() + 3)).pow(2).sum(1, keepdim=True) + n) + 2
    lp = d - ln
    dlp = U32 * (rel + 2 * ln.abs() + d.abs() + lp.abs())
    dU = torch.sqrt((p * d * (2 * d.abs() + 5)).pow(2).sum(1, keepdim=True) + n * U.pow(2)) + 2 * U.abs()
    H = ln - U
    dH = U32 * (rel * (1 + U.abs()) + dU + 2 * ln.abs() + 2 * U.abs() + H.abs())
    return lp, H[:, 0], dlp.pow(2).mean(), dH.pow(2).mean()
