"""The FP8 operators' definitions in float64 (torch, on whatever device the
inputs are), the inputs of their tests, and error bounds by counting
roundings.  U32 is half a step of fp32 relative to the value, and so on."""

import torch

RUN = 128
U32, UBF16, UE4M3 = 2.0 ** -24, 2.0 ** -8, 2.0 ** -4
E4M3_TINY = 2.0 ** -10            # half a step of E4M3's subnormals
SCALE_MIN = 2.0 ** -126
# The fp8 matrix instruction aligns the 128 products of a step to the largest
# of them and cuts them off 16 bits below it: each loses less than 2^-16 of it
# (measured over ten million sums of wide values: at most 2^-9.4 in all).
FAST_STEP = 128 * 2.0 ** -16


def runs(n):
    return (n + RUN - 1) // RUN


def rows64(codes, scales):
    """Token rows as values: [rows][K]."""
    K = codes.shape[-1]
    return codes.double() * scales.double().repeat_interleave(RUN, -1)[..., :K]


def blocks64(codes, scales):
    """A weight matrix as values: [N][K]."""
    N, K = codes.shape
    return codes.double() * scales.double().repeat_interleave(RUN, 0)[:N].repeat_interleave(RUN, 1)[:, :K]


def product(a, a_s, w, w_s, fast=False):
    """(out, bound): the product in float64 and how far an fp32 evaluation in
    steps of 128 may be off: a step's 128 exact products added in fp32 (at
    most 127 roundings), one rounding of the factor as * ws, and one per step
    and per partial sum over the steps (at most S + 8).  fast: the fp8
    instruction's alignment on top, from each step's largest product."""
    av, wv = rows64(a, a_s), blocks64(w, w_s)
    out = av @ wv.t().contiguous()
    S = runs(a.shape[1])
    bound = (127 + 1 + S + 8) * U32 * (av.abs() @ wv.abs().t().contiguous())
    if fast:
        for s in range(S):
            k = slice(s * RUN, (s + 1) * RUN)
            bound += FAST_STEP * torch.outer(av[:, k].abs().amax(1), wv[:, k].abs().amax(1))
    return out, bound


def check_rounded(got, want, bound, dtype, what=""):
    """got is within `bound` and one rounding to its type of `want`."""
    u = {torch.float32: U32, torch.bfloat16: UBF16}[dtype]
    assert got.dtype == dtype, what
    err = (got.double() - want).abs()
    lim = bound + u * (want.abs() + bound)
    assert torch.isfinite(got.double()).all(), f"{what}: non-finite"
    over = err - lim
    assert (over <= 0).all(), f"{what}: off by {float(err.max()):.3e}, worst over the bound {float(over.max()):.3e}"


def check_quantised(q, scales, v, dv, what=""):
    """Codes and scales of v (float64), each value of which the kernel knows
    to within dv (a tensor): scale max|v| / 448 (one rounding more), codes the
    nearest E4M3 to v / scale (one division's rounding more)."""
    rows, n = v.shape
    pad = runs(n) * RUN - n
    vp = torch.nn.functional.pad(v, (0, pad)).view(rows, -1, RUN).abs()
    dp = torch.nn.functional.pad(dv, (0, pad)).view(rows, -1, RUN)
    lo, hi = (vp - dp).amax(-1) / 448.0, (vp + dp).amax(-1) / 448.0
    s = scales.double()
    assert scales.dtype == torch.float32 and s.shape == lo.shape, what
    assert (s >= torch.clamp(lo * (1 - 2 * U32), min=SCALE_MIN * (1 - U32))).all(), f"{what}: a scale is too small"
    assert (s <= torch.clamp(hi * (1 + 2 * U32), min=SCALE_MIN * (1 + U32))).all(), f"{what}: a scale is too large"
    each = s.repeat_interleave(RUN, 1)[:, :n]
    want = v / each
    err = (q.double() - want).abs()
    known = dv / each + 2 * U32 * want.abs()
    lim = UE4M3 * (want.abs() + known) + E4M3_TINY + known
    assert torch.isfinite(q.double()).all(), f"{what}: non-finite codes"
    assert (err <= lim).all(), f"{what}: a code is off by {float((err - lim).max()):.3e} more than half a step"


def norm(x, residual, weight, eps):
    """(h as stored, v, dv): the residual's addition rounded to its type, and
    the norm of what is stored with its relative error counted: the sum of
    squares (8 per chunk of 2048 columns and thread, then 6 + 4 partial sums,
    squares not rounded apart; more threads add at most 12 partial sums and
    save 8 or more per chunk past the first), half of that through the root, four roundings
    for mean, eps, root and inverse, two products."""
    if residual is not None:
        h = (x.float() + residual.float()).to(residual.dtype)
    else:
        h = x
    hd = h.double()
    d = x.shape[1]
    v = hd / torch.sqrt((hd * hd).mean(1, keepdim=True) + eps)
    if weight is not None:
        v = v * weight.double()
    chunks = (d + 2047) // 2048
    return h, v, (0.5 * (8 * chunks + 10) + 6) * U32 * v.abs()


def gate_up(a, a_s, g, g_s, u, u_s):
    """(v, dv) of silu(g a) * (u a) for rows of one expert."""
    gv, dg = product(a, a_s, g, g_s)
    uv, du = product(a, a_s, u, u_s)
    silu = gv * torch.sigmoid(gv)
    v = silu * uv
    # |silu'| <= 1.1; exp, sum, division and two products: exp's argument is
    # exact and its result good to 2 units, so 8 roundings cover them
    return v, 1.1 * dg * (uv.abs() + du) + silu.abs() * du + 8 * U32 * v.abs()


# ---------------------------------------------------------------- inputs

def gen(seed, dev="cuda"):
    return torch.Generator(device=dev).manual_seed(seed)


def codes(g, *shape, dev="cuda"):
    return (112 * torch.randn(shape, generator=g, device=dev)).clamp(-448, 448).to(torch.float8_e4m3fn)


def scales(g, *shape, dev="cuda", mean=2.0 ** -9):
    return mean * torch.exp2(4 * torch.rand(shape, generator=g, device=dev) - 2)


def routing(g, T, E, k, dev="cuda", only=None):
    """offsets, perm and ids of k distinct experts per token (`only`: from
    these experts)."""
    pick = torch.arange(E, device=dev) if only is None else torch.tensor(only, device=dev)
    ids = pick[torch.rand((T, len(pick)), generator=g, device=dev).topk(k, dim=1).indices].reshape(-1)
    perm = torch.sort(ids, stable=True).indices
    off = torch.cat([ids.new_zeros(1), torch.bincount(ids, minlength=E).cumsum(0)])
    return off.to(torch.int32), perm.to(torch.int32), ids
