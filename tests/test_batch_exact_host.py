"""The inputs of tests/batch_exact.py on the CPU: the definitions give the results
that they claim, and a mistake planted in them does not pass."""

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
