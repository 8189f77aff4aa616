"""The entry points of a batch of many requests on the host (no GPU needed):
every invalid request is rejected with the documented status before any HIP
call, and empty calls enqueue nothing."""

import pytest

import quantized_routed_moe_amd as qm

A = 0x10000            # fake, 16-byte aligned "device" address (never dereferenced)
BF16, F32 = qm.MOE_TYPE_BF16, qm.MOE_TYPE_F32
BIG = 1 << 62


def plan(T=100, L=8, ids=A, off=A, perm=A, items=A, ws=A, n=BIG):
    return qm.lib().moe_lora_plan(T, L, ids, off, perm, items, ws, n, None)


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), qm.MOE_ERR_SHAPE), (dict(T=1 << 26), qm.MOE_ERR_SHAPE), (dict(L=0), qm.MOE_ERR_SHAPE),
    (dict(L=1025), qm.MOE_ERR_SHAPE), (dict(L=-3), qm.MOE_ERR_SHAPE),
    *[(dict([(n, None)]), qm.MOE_ERR_NULL) for n in ("ids", "off", "perm", "items")],
    *[(dict([(n, A + 2)]), qm.MOE_ERR_ALIGN) for n in ("ids", "off", "perm", "items")],
    (dict(items=A + 8), qm.MOE_ERR_ALIGN), (dict(T=8193, ws=None), qm.MOE_ERR_NULL),
    (dict(T=8193, ws=A + 4), qm.MOE_ERR_ALIGN), (dict(T=8193, n=4 * 9 * 3 - 1), qm.MOE_ERR_WORKSPACE),
])
def test_plan_refusals(over, code):
    assert plan(**over) == code


def test_plan_sizes():
    L = qm.lib()
    assert plan(T=0, ids=None, off=None, perm=None, items=None, ws=None, n=0) == qm.MOE_OK
    # each group's last run as short as can be
    assert [L.moe_lora_items(T, 8) for T in (0, 1, 2, 9, 10, 64, 100, 640)] == [0, 1, 2, 9, 9, 9, 10, 18]
    assert L.moe_lora_items(-1, 8) == 0 and L.moe_lora_items(5, 0) == 0 and L.moe_lora_items(5, 1025) == 0
    wb = L.moe_lora_plan_workspace_bytes
    assert wb(0, 8) == wb(8192, 1024) == wb(-1, 8) == wb(1 << 26, 8) == wb(9000, 0) == 0
    assert wb(8193, 8) == 256 and wb(8193, 1024) == (3 * 1025 * 4 + 255) // 256 * 256


def lora(T=4, K=64, N=100, r=16, L=8, x=A, xs=64, a=A, b=A, sc=A, perm=A, items=A, base=A, bs=100, out=2 * A, os=100, ty=BF16,
         ws=A, n=BIG):
    return qm.lib().moe_lora_add(T, K, N, r, L, x, xs, a, b, sc, perm, items, base, bs, out, os, ty, ws, n, None)


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), qm.MOE_ERR_SHAPE), (dict(T=1 << 26), qm.MOE_ERR_SHAPE), (dict(K=0), qm.MOE_ERR_SHAPE),
    (dict(K=48, xs=48), qm.MOE_ERR_SHAPE), (dict(K=(1 << 22) + 32, xs=1 << 23), qm.MOE_ERR_SHAPE), (dict(N=0), qm.MOE_ERR_SHAPE),
    (dict(N=1 << 30), qm.MOE_ERR_SHAPE), (dict(r=0), qm.MOE_ERR_SHAPE), (dict(r=12), qm.MOE_ERR_SHAPE), (dict(r=264), qm.MOE_ERR_SHAPE),
    (dict(L=0), qm.MOE_ERR_SHAPE), (dict(L=1025), qm.MOE_ERR_SHAPE),
    (dict(xs=63), qm.MOE_ERR_SHAPE), (dict(xs=68), qm.MOE_ERR_SHAPE), (dict(xs=32), qm.MOE_ERR_SHAPE), (dict(xs=-64), qm.MOE_ERR_SHAPE),
    (dict(xs=1 << 41), qm.MOE_ERR_SHAPE), (dict(bs=99), qm.MOE_ERR_SHAPE), (dict(os=99), qm.MOE_ERR_SHAPE), (dict(os=0), qm.MOE_ERR_SHAPE),
    (dict(bs=-100), qm.MOE_ERR_SHAPE), (dict(os=1 << 41), qm.MOE_ERR_SHAPE),
    (dict(T=(1 << 26) - 1, N=1 << 12, bs=1 << 12, os=1 << 12), qm.MOE_ERR_SHAPE),
    (dict(T=(1 << 26) - 1, r=256), qm.MOE_ERR_SHAPE),                                  # of those that make v
    (dict(T=1 << 22, N=1 << 20, bs=1 << 20, os=1 << 20), qm.MOE_ERR_SHAPE),            # more workgroups than a grid has
    *[(dict([(n, None)]), qm.MOE_ERR_NULL) for n in ("x", "a", "b", "perm", "items", "base", "out")],
    *[(dict([(n, A + 8)]), qm.MOE_ERR_ALIGN) for n in ("x", "a", "b", "items", "base", "out")],
    *[(dict([(n, A + 2)]), qm.MOE_ERR_ALIGN) for n in ("perm", "sc")],
    (dict(ty=0), qm.MOE_ERR_FORMAT), (dict(ty=3), qm.MOE_ERR_FORMAT), (dict(out=A, os=104), qm.MOE_ERR_UNSUPPORTED),
    (dict(out=A, bs=0), qm.MOE_ERR_UNSUPPORTED), (dict(T=10000, ws=None), qm.MOE_ERR_NULL),
    (dict(T=10000, ws=A + 8), qm.MOE_ERR_ALIGN), (dict(T=10000, n=10000 * 16 * 4 - 1), qm.MOE_ERR_WORKSPACE),
])
def test_lora_refusals(over, code):
    assert lora(**over) == code


def test_lora_of_no_tokens():
    assert lora(T=0, x=None, a=None, b=None, perm=None, items=None, base=None, out=None, ws=None, n=0) == qm.MOE_OK
    wb = qm.lib().moe_lora_add_workspace_bytes
    assert wb(0, 64, 100, 16, 8) == 0 and wb(4, 64, 100, 12, 8) == 0 and wb(10000, 64, 100, 16, 8) >= 10000 * 16 * 4


def scores(T=4, V=1000, l=A, ty=BF16, st=1000, tok=A, given=1, lp=A, ent=A, top=5, ids=A, tlp=A, ws=A, n=BIG):
    return qm.lib().moe_token_logprobs(T, V, l, ty, st, tok, given, lp, ent, top, ids, tlp, ws, n, None)


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), qm.MOE_ERR_SHAPE), (dict(T=1 << 30), qm.MOE_ERR_SHAPE), (dict(V=0), qm.MOE_ERR_SHAPE),
    (dict(V=1 << 30, st=1 << 30), qm.MOE_ERR_SHAPE), (dict(given=-1), qm.MOE_ERR_SHAPE), (dict(given=4097), qm.MOE_ERR_SHAPE),
    (dict(top=-1), qm.MOE_ERR_SHAPE), (dict(top=65), qm.MOE_ERR_SHAPE), (dict(V=4, top=5), qm.MOE_ERR_SHAPE),
    (dict(st=999), qm.MOE_ERR_SHAPE), (dict(st=0), qm.MOE_ERR_SHAPE), (dict(st=1 << 41), qm.MOE_ERR_SHAPE),
    *[(dict([(n, None)]), qm.MOE_ERR_NULL) for n in ("l", "tok", "lp", "ids", "tlp")],
    (dict(given=0, top=0, ent=None), qm.MOE_ERR_NULL), (dict(ty=0), qm.MOE_ERR_FORMAT), (dict(l=A + 8), qm.MOE_ERR_ALIGN),
    *[(dict([(n, A + 2)]), qm.MOE_ERR_ALIGN) for n in ("tok", "lp", "ent", "ids", "tlp")],
    (dict(T=1, V=100000, st=100000, ws=None), qm.MOE_ERR_NULL), (dict(T=1, V=100000, st=100000, ws=A + 8), qm.MOE_ERR_ALIGN),
    (dict(T=1, V=100000, st=100000, n=64), qm.MOE_ERR_WORKSPACE),
])
def test_scores_refusals(over, code):
    assert scores(**over) == code


def test_scores_of_no_rows():
    assert scores(T=0, l=None, tok=None, lp=None, ent=None, ids=None, tlp=None, ws=None, n=0) == qm.MOE_OK
    wb = qm.lib().moe_token_logprobs_workspace_bytes
    assert wb(0, 1000, 5) == wb(-1, 1000, 5) == wb(4, 1000, 65) == wb(2048, 128256, 5) == 0 and wb(1, 128256, 5) > 0


def test_python_takes_device_tensors_only():
    import torch
    ids = torch.zeros(4, dtype=torch.int32)
    x, a, b = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((2, 8, 64), dtype=torch.bfloat16), torch.zeros((2, 16, 8), dtype=torch.bfloat16)
    base = torch.zeros((4, 16), dtype=torch.bfloat16)
    for call in (lambda: qm.lora_plan(ids, 2), lambda: qm.token_logprobs(base),
                 lambda: qm.lora_add(base, x, a, b, qm.LoraPlan(4, 2, ids, ids, ids))):
        with pytest.raises(ValueError, match="device tensors"):
            call()
