"""Inputs of the operators of a batch of many requests whose results are known to
the bit: what a bound that counts the worst
roundings of long sums would let through shows there (torch, on whatever device
the generator is)."""

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
