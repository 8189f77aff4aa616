"""The operators of a batch of many requests on the GPU at inputs whose results are
known to the bit (tests/batch_exact.py): all 24 bits of v on every way that hands it
over, and every value of a row on every way that takes it; and the mean square of
the errors of ordinary inputs."""

import pytest
import torch

import batch_exact as X
import batch_ref as B
import quantized_routed_moe_amd as qm
from batch_ref import gen

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


# ------------------------------------------------------------------ adapters

# few tokens without a workspace, and one to eight steps of 32 ranks; columns in whole 16 bytes or not
@pytest.mark.parametrize("N", [520, 1111])
@pytest.mark.parametrize("K,r", [(96, 8), (96, 32), (1056, 16), (4096, 24), (1056, 40), (4096, 64), (416, 72), (4096, 128), (1056, 136),
                                 (4096, 256)])
@pytest.mark.parametrize("T,L", [(1, 1), (2, 1), (4, 3), (5, 2), (17, 1), (33, 2), (150, 40), (700, 6)])
def test_v_has_24_bits(T, L, K, r, N):
    g = gen(T + K + r + N)
    ids = torch.randint(-1 if T > 2 else 0, L, (T,), generator=g, device="cuda", dtype=I32)
    base, x, a, b, s, out = X.lora_case(g, T, K, N, r, L, ids)
    plan = qm.lora_plan(ids, L)
    assert torch.equal(qm.lora_add(base, x, a, b, plan, scales=s), out)
    got = qm.lora_add(base.to(BF16), x, a, b, plan, scales=s)
    assert torch.equal(got, out.to(BF16))


@pytest.mark.parametrize("K,r,L,run", [(4096, 32, 16, 256), (4096, 128, 16, 256), (2080, 256, 4, 700)])
def test_v_of_many_tokens_has_24_bits(K, r, L, run):
    T, N = 2048, 1032
    g = gen(K + r)
    ids = torch.randint(0, L, (T // run + 1,), generator=g, device="cuda", dtype=I32).repeat_interleave(run)[:T].contiguous()
    base, x, a, b, s, out = X.lora_case(g, T, K, N, r, L, ids)
    assert torch.equal(qm.lora_add(base, x, a, b, qm.lora_plan(ids, L), scales=s), out)


@pytest.mark.parametrize("T,K,r,waves", [(1, 4096, 16, 8), (4, 2048, 16, 8), (64, 4096, 16, 4), (300, 4096, 64, 4), (64, 2048, 128, 4),
                                         (500, 1024, 256, 4)])
def test_mean_square_of_the_error_of_v(T, K, r, waves):
    """Ordinary inputs, each column one rank: the error of v is that of an fp32 sum."""
    g = gen(T + K)
    x, a, _, _, _ = B.lora_case(g, T, K, 1, r, 2, F32)
    b = torch.eye(r, device="cuda").to(BF16).expand(2, r, r).contiguous()
    ids = torch.randint(0, 2, (T,), generator=g, device="cuda", dtype=I32)
    got = qm.lora_add(torch.zeros((T, r), device="cuda"), x, a, b, qm.lora_plan(ids, 2))
    want = torch.empty((T, r), dtype=torch.float64, device="cuda")
    for e in (0, 1):
        t = torch.nonzero(ids == e)[:, 0]
        want[t] = x[t].double() @ a[e].double().t().contiguous()
    err = (got.double() - want).pow(2).mean() / want.pow(2).mean()
    assert float(err) <= X.sum_bound(K, waves), float(err)


@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("values,halves", [(2, 2 ** 1.5), (32, 4 * 2 ** 1.5 + 2)])
def test_dot_products_of_few_tokens(T, values, halves):
    """A dot product of two values and what is there is off by at most 2^1.5 halves of the
    magnitudes; of 32 values a lane takes four, and two sums join the lanes."""
    K, r = 32, 16
    worst = 0.0
    for seed in range(40):
        g = gen(seed)
        size = torch.exp2(torch.randint(-12, 13, (K,), generator=g, device="cuda").float())
        x = torch.zeros((T, K), device="cuda")
        at = 0 if values == K else int(torch.randint(0, K // 2, (1,), generator=g, device="cuda")) * 2
        x[:, at:at + values] = (torch.randn((T, K), generator=g, device="cuda") * size)[:, at:at + values]
        x = x.to(BF16)
        a = torch.randn((1, r, K), generator=g, device="cuda").to(BF16)
        b = torch.eye(r, device="cuda").to(BF16)[None].contiguous()
        got = qm.lora_add(torch.zeros((T, r), device="cuda"), x, a, b, qm.lora_plan(torch.zeros(T, dtype=I32, device="cuda"), 1))
        p = x.double()[:, None, :] * a.double()
        over = (got.double() - p.sum(2)).abs() / (X.U32 * p.abs().sum(2))
        worst = max(worst, float(over.max()))
    assert worst <= halves, worst


@pytest.mark.parametrize("T", [1, 3, 5, 40])
@pytest.mark.parametrize("scale", [-58, -62, -70])
def test_values_below_the_normal_range(T, scale):
    """v of about 2^-116, 2^-124 and 2^-140 and columns that make much of them: lost are at
    most 2^-126 for each product and each part of a v."""
    K, N, r, L = 96, 40, 24, 2
    g = gen(T - scale)
    x, a, b, base, s = B.lora_case(g, T, K, N, r, L, F32)
    x, a, b = x * 2.0 ** scale, a * 2.0 ** scale, b * 2.0 ** 100
    ids = torch.randint(0, L, (T,), generator=g, device="cuda", dtype=I32)
    base.zero_()
    got = qm.lora_add(base, x, a, b, qm.lora_plan(ids, L), scales=s)
    want, bound = B.lora(base, x, a, b, ids, s)
    lost = (K + 3) * b[ids.long()].double().abs().sum(2) * s[ids.long()].double()[:, None] * 2.0 ** -126
    B.check_rounded(got, want, bound + lost, F32)
    if scale == -58:
        assert float((want.abs() / lost).median()) > 1          # the results are not lost in it


# -------------------------------------------------------------------- scores

# a row a wave; a row a workgroup; seen twice, held and read again; parts of a row, held and read again
WAYS = [(2051, 4096, BF16), (2050, 1023, F32), (2048, 15, BF16), (600, 333, BF16), (700, 5003, BF16), (1300, 20011, BF16),
        (700, 16001, BF16), (640, 8003, F32), (9, 50001, BF16), (17, 128256, BF16), (9, 128257, F32), (77, 50001, BF16), (9, 1050001, BF16),
        (9, 600011, F32)]


@pytest.mark.parametrize("kind", ["all", "half", "few", "ends", "chunks"])
@pytest.mark.parametrize("T,V,dtype", WAYS)
def test_every_value_of_a_row_counts_once(T, V, dtype, kind):
    """Rows that begin at every place of 16 bytes, with what lies between them larger than
    all of theirs."""
    g = gen(T + V)
    per = 8 if dtype == BF16 else 4
    here, l = X.counted(g, T, V, dtype, kind, per)
    step = V // per * per + per + 1
    buf = torch.full((T, step), 1e6, device="cuda").to(dtype)
    buf[:, :V] = l
    tok = torch.cat([here.float().argmax(1, keepdim=True), torch.randint(0, V, (T, 2), generator=g, device="cuda")], 1).to(I32)
    for top in (0, 3, 30):
        top = min(top, V)
        got = qm.token_logprobs(buf[:, :V], tok, top=top, entropy=top != 3)
        X.check_counted(here, l, tok, top, got, f"top {top}")


@pytest.mark.parametrize("T,V,dtype", [(64, 128256, BF16), (64, 128256, F32), (300, 50001, F32), (1300, 20011, BF16), (2048, 2048, F32)])
def test_mean_square_of_the_errors_of_scores(T, V, dtype):
    g = gen(T)
    l = (2.5 * torch.randn((T, V), generator=g, device="cuda")).to(dtype)
    tok = torch.randint(0, V, (T, 8), generator=g, device="cuda", dtype=I32)
    lp, ent, _, _ = qm.token_logprobs(l, tok, entropy=True)
    e_lp, e_h = [], []
    b_lp = b_h = 0.0
    for t in range(0, T, 256):
        want, H, dlp, dH = X.scores_mean_square(l[t:t + 256])
        e_lp.append((lp[t:t + 256].double() - want.gather(1, tok[t:t + 256].long())).pow(2).flatten())
        e_h.append((ent[t:t + 256].double() - H).pow(2))
        b_lp, b_h = max(b_lp, float(dlp)), max(b_h, float(dH))
    assert float(torch.cat(e_lp).mean()) <= b_lp and float(torch.cat(e_h).mean()) <= b_h
