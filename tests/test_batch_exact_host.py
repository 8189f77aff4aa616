"""The inputs of tests/batch_exact.py on the CPU: the definitions give the results
that they claim, and a mistake planted in them does not pass."""

import math

import pytest
import torch

import batch_exact as X
import batch_ref as B

F32 = torch.float32


def cpu(seed):
    return torch.Generator().manual_seed(seed)


def ids_of(g, T, L):
    return torch.randint(-1, L, (T,), generator=g, dtype=torch.int32)


@pytest.mark.parametrize("T,K,N,r,L", [(5, 96, 33, 32, 2), (40, 1056, 300, 64, 4), (17, 4096, 520, 256, 3)])
def test_adapters_are_exact(T, K, N, r, L):
    g = cpu(T)
    ids = ids_of(g, T, L)
    base, x, a, b, s, out = X.lora_case(g, T, K, N, r, L, ids)
    want, _ = B.lora(base, x, a, b, ids, s)
    assert torch.equal(want, out.double())
    # fp32 sums in another order are exact too
    for t in range(T):
        if ids[t] >= 0:
            v = torch.zeros(r)
            for k in torch.randperm(K, generator=g).tolist():
                if a[ids[t], :, k].any():
                    v += x[t, k].float() * a[ids[t], :, k].float()
            assert torch.equal((b[ids[t]].float() @ v) * s[ids[t]], out[t])
            break


@pytest.mark.parametrize("T,K,N,r,L", [(2, 96, 33, 8, 1), (40, 1056, 300, 64, 4)])
def test_fewer_parts_of_v_do_not_pass(T, K, N, r, L):
    """Three bf16 parts hold a v; with two nearly every value is another, with one all are."""
    g = cpu(T + 1)
    ids = torch.randint(0, L, (T,), generator=g, dtype=torch.int32)
    base, x, a, b, s, out = X.lora_case(g, T, K, N, r, L, ids)
    v = torch.stack([a[e].double() @ x[t].double() for t, e in enumerate(ids.tolist())]).float()

    def result(parts):
        w = X.in_parts(v, parts)
        return torch.stack([(b[e].double() @ w[t].double()) * s[e].double() for t, e in enumerate(ids.tolist())]).float()

    assert torch.equal(result(3), out)
    assert float((result(2) != out).float().mean()) > 0.9 and float((result(1) != out).float().mean()) > 0.9


def test_mean_square_bound_excludes_fewer_parts():
    v = torch.randn(100000, generator=cpu(5))
    for parts, inside in ((3, True), (2, False), (1, False)):
        e = (X.in_parts(v, parts) - v).double().pow(2).mean() / v.double().pow(2).mean()
        assert (float(e) <= X.sum_bound(4096, 4)) == inside


def answers(here, logits, tokens, top, seen=None):
    """What token_logprobs would give if it summed the places `seen`."""
    seen = here if seen is None else seen
    ln = torch.log(seen.sum(1).double())[:, None]
    lp = torch.where(here, 0.0, torch.where(torch.isinf(logits), -math.inf, -X.LOW)).double() - ln
    order = torch.sort(~here, dim=1, stable=True).indices[:, :top]
    return lp.gather(1, tokens.long()).float(), ln[:, 0].float(), order.to(torch.int32), lp.gather(1, order).float()


@pytest.mark.parametrize("V", [100, 4096, 50001, 128256])
@pytest.mark.parametrize("kind", ["all", "half", "few", "ends", "chunks"])
def test_a_value_too_many_or_too_few_does_not_pass(kind, V):
    g = cpu(V)
    T, per = 6, 8
    here, logits = X.counted(g, T, V, F32, kind, per)
    tokens = torch.cat([here.float().argmax(1, keepdim=True), torch.randint(0, V, (T, 1), generator=g)], 1)
    X.check_counted(here, logits, tokens, 7, answers(here, logits, tokens, 7))
    for less in (1, 8):
        seen = here.clone()
        row = int(here.sum(1).argmax())
        seen[row, torch.nonzero(here[row])[-less:, 0]] = False
        if not seen[row].any():
            continue
        for what, got in (("logprobs", 0), ("entropy", 1)):
            bad = list(answers(here, logits, tokens, 7))
            bad[got] = answers(here, logits, tokens, 7, seen)[got]
            with pytest.raises(AssertionError, match=what):
                X.check_counted(here, logits, tokens, 7, bad)
