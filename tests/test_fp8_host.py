"""The FP8 entry points on the host (no GPU needed): every invalid request is
rejected with the documented status before any HIP call, and empty calls
enqueue nothing."""

import ctypes

import pytest

import quantized_routed_moe_amd as qm

A = 0x10000            # fake, 16-byte aligned "device" address (never dereferenced)
BF16, F32 = qm.MOE_TYPE_BF16, qm.MOE_TYPE_F32


def norm(T=4, d=256, x=A, xt=BF16, xs=256, res=A, ro=2 * A, rt=BF16, rs=256, ros=256, w=A, wt=BF16, eps=1e-6, y=A, q=A,
         sc=A):
    return qm.lib().moe_add_rmsnorm(T, d, x, xt, xs, res, ro, rt, rs, ros, w, wt, eps, y, q, sc, None)


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), qm.MOE_ERR_SHAPE), (dict(d=0), qm.MOE_ERR_SHAPE), (dict(d=48), qm.MOE_ERR_SHAPE),
    (dict(d=(1 << 20) + 32), qm.MOE_ERR_SHAPE), (dict(eps=-1.0), qm.MOE_ERR_SHAPE),
    (dict(eps=float("nan")), qm.MOE_ERR_SHAPE), (dict(eps=float("inf")), qm.MOE_ERR_SHAPE),
    (dict(x=None), qm.MOE_ERR_NULL), (dict(res=None), qm.MOE_ERR_NULL), (dict(ro=None), qm.MOE_ERR_NULL),
    (dict(q=None), qm.MOE_ERR_NULL), (dict(sc=None), qm.MOE_ERR_NULL),
    (dict(res=None, ro=None, y=None, q=None, sc=None), qm.MOE_ERR_NULL),
    (dict(xt=0), qm.MOE_ERR_FORMAT), (dict(rt=3), qm.MOE_ERR_FORMAT), (dict(wt=7), qm.MOE_ERR_FORMAT),
    (dict(xs=260), qm.MOE_ERR_SHAPE), (dict(xs=128), qm.MOE_ERR_SHAPE), (dict(xs=-256), qm.MOE_ERR_SHAPE),
    (dict(rs=250), qm.MOE_ERR_SHAPE), (dict(ros=0), qm.MOE_ERR_SHAPE), (dict(ros=248), qm.MOE_ERR_SHAPE),
    (dict(xt=F32, xs=258), qm.MOE_ERR_SHAPE), (dict(xs=1 << 41), qm.MOE_ERR_SHAPE),
    (dict(ro=A, rs=512), qm.MOE_ERR_UNSUPPORTED),
    (dict(x=A + 8), qm.MOE_ERR_ALIGN), (dict(ro=A + 4), qm.MOE_ERR_ALIGN), (dict(w=A + 2), qm.MOE_ERR_ALIGN),
    (dict(y=A + 2), qm.MOE_ERR_ALIGN), (dict(q=A + 1), qm.MOE_ERR_ALIGN), (dict(sc=A + 2), qm.MOE_ERR_ALIGN),
])
def test_norm_refusals(over, code):
    assert norm(**over) == code


def test_norm_of_no_rows():
    assert norm(T=0, x=None, res=None, ro=None, y=None, q=None, sc=None) == qm.MOE_OK


def gemm(M=4, N=100, K=256, a=A, sa=256, asc=A, w=A, wsc=A, out=A, ot=BF16, so=100):
    return qm.lib().moe_gemm_fp8(M, N, K, a, sa, asc, w, wsc, out, ot, so, None)


@pytest.mark.parametrize("over,code", [
    (dict(M=-1), qm.MOE_ERR_SHAPE), (dict(N=0), qm.MOE_ERR_SHAPE), (dict(K=0), qm.MOE_ERR_SHAPE),
    (dict(K=40), qm.MOE_ERR_SHAPE), (dict(M=1 << 30), qm.MOE_ERR_SHAPE), (dict(N=1 << 30), qm.MOE_ERR_SHAPE),
    (dict(M=(1 << 30) - 1, N=(1 << 30) - 1, so=1 << 30), qm.MOE_ERR_SHAPE),       # more workgroups than a grid has
    (dict(a=None), qm.MOE_ERR_NULL), (dict(asc=None), qm.MOE_ERR_NULL), (dict(w=None), qm.MOE_ERR_NULL),
    (dict(wsc=None), qm.MOE_ERR_NULL), (dict(out=None), qm.MOE_ERR_NULL), (dict(ot=0), qm.MOE_ERR_FORMAT),
    (dict(sa=240), qm.MOE_ERR_SHAPE), (dict(sa=264), qm.MOE_ERR_SHAPE), (dict(so=99), qm.MOE_ERR_SHAPE),
    (dict(a=A + 8), qm.MOE_ERR_ALIGN), (dict(w=A + 8), qm.MOE_ERR_ALIGN), (dict(out=A + 8), qm.MOE_ERR_ALIGN),
    (dict(asc=A + 2), qm.MOE_ERR_ALIGN), (dict(wsc=A + 2), qm.MOE_ERR_ALIGN),
])
def test_gemm_refusals(over, code):
    assert gemm(**over) == code


def grouped(R=8, E=4, N=64, K=128, a=A, rows=4, asc=A, w=A, wsc=A, off=A, perm=A, k=2, out=A, ot=F32):
    return qm.lib().moe_grouped_gemm_fp8(R, E, N, K, a, rows, asc, w, wsc, off, perm, k, out, ot, None)


@pytest.mark.parametrize("over,code", [
    (dict(R=-1), qm.MOE_ERR_SHAPE), (dict(E=0), qm.MOE_ERR_SHAPE), (dict(E=65), qm.MOE_ERR_SHAPE),
    (dict(N=0), qm.MOE_ERR_SHAPE), (dict(K=100), qm.MOE_ERR_SHAPE), (dict(k=0), qm.MOE_ERR_SHAPE),
    (dict(rows=0), qm.MOE_ERR_SHAPE), (dict(perm=None), qm.MOE_ERR_SHAPE),        # 8 rows of a are needed without perm
    (dict(a=None), qm.MOE_ERR_NULL), (dict(off=None), qm.MOE_ERR_NULL), (dict(out=None), qm.MOE_ERR_NULL),
    (dict(ot=5), qm.MOE_ERR_FORMAT), (dict(off=A + 2), qm.MOE_ERR_ALIGN), (dict(perm=A + 1), qm.MOE_ERR_ALIGN),
    (dict(out=A + 4), qm.MOE_ERR_ALIGN),
])
def test_grouped_refusals(over, code):
    assert grouped(**over) == code


def test_empty_products():
    assert gemm(M=0, a=None, out=None) == qm.MOE_OK
    assert grouped(R=0, a=None, off=None, out=None) == qm.MOE_OK


def shape(T=4, d=256, E=8, k=2, f=128):
    return qm.moe_shape(T, d, E, k, f)


def gate_up(s=None, ws=A, n=1 << 30, **over):
    p = dict(a=A, asc=A, gate=A, gsc=A, up=A, usc=A, off=A, perm=A, act=A, actsc=A)
    p.update(over)
    return qm.lib().moe_expert_gate_up_fp8(ctypes.byref(s or shape()), *p.values(), ws, n, None)


@pytest.mark.parametrize("over,code", [
    (dict(s=shape(k=9)), qm.MOE_ERR_SHAPE), (dict(s=shape(d=48)), qm.MOE_ERR_SHAPE), (dict(s=shape(E=65)), qm.MOE_ERR_SHAPE),
    *[(dict([(n, None)]), qm.MOE_ERR_NULL) for n in ("a", "asc", "gate", "gsc", "up", "usc", "off", "perm", "act", "actsc")],
    *[(dict([(n, A + 8)]), qm.MOE_ERR_ALIGN) for n in ("a", "gate", "up", "act", "ws")],
    *[(dict([(n, A + 2)]), qm.MOE_ERR_ALIGN) for n in ("asc", "gsc", "usc", "off", "perm", "actsc")],
    (dict(ws=None), qm.MOE_ERR_NULL), (dict(n=8 * 128 * 4 - 1), qm.MOE_ERR_WORKSPACE),
])
def test_gate_up_refusals(over, code):
    assert gate_up(**over) == code


def test_workspace_sizes():
    al = lambda v: (v + 255) // 256 * 256  # noqa: E731
    wb = lambda s: qm.lib().moe_expert_gate_up_fp8_workspace_bytes(ctypes.byref(s))  # noqa: E731
    # fp32 silu(g) u of every row, and an 8-byte flag per 16 columns and run
    # of 16 rows: at most 8 / 16 + min(E, 8) runs
    few = al(8 * 128 * 4) + al(8 * 8 * 8)
    assert wb(shape()) == few
    assert wb(shape(T=2048, d=4096, E=64, f=2048)) == 0   # workgroups of whole runs need none
    assert wb(shape(k=0)) == 0 and wb(shape(T=0)) == 0
    assert gate_up(s=shape(T=0), ws=None, n=0) == qm.MOE_OK
    assert gate_up(n=few - 1) == qm.MOE_ERR_WORKSPACE
    lw = lambda s: qm.lib().moe_layer_fp8_workspace_bytes(ctypes.byref(s))  # noqa: E731
    assert lw(shape()) == 256 + al(9 * 4) + 2 * al(8 * 4) + al(8 * 128) + al(8 * 4) + few + al(8 * 256 * 4)
    assert lw(shape(f=100)) == 0


def layer(s=None, x=A, xq=A, xs=A, wr=A, bias=None, logits=A, ids=A, w=A, out=A, ws=A, n=1 << 30, ex=True, **over):
    e = qm.moe_fp8_experts(A, A, A, A, A, A)
    for k, v in over.items():
        setattr(e, k, v)
    return qm.lib().moe_layer_fp8(ctypes.byref(s or shape()), x, xq, xs, wr, bias, logits,
                                  ctypes.byref(e) if ex else None, ids, w, out, ws, n, None)


@pytest.mark.parametrize("over,code", [
    (dict(s=shape(E=0)), qm.MOE_ERR_SHAPE), (dict(x=None), qm.MOE_ERR_NULL), (dict(xq=None), qm.MOE_ERR_NULL),
    (dict(xs=None), qm.MOE_ERR_NULL), (dict(logits=None), qm.MOE_ERR_NULL), (dict(ids=None), qm.MOE_ERR_NULL),
    (dict(out=None), qm.MOE_ERR_NULL), (dict(ws=None), qm.MOE_ERR_NULL), (dict(ex=False), qm.MOE_ERR_NULL),
    (dict(down=None), qm.MOE_ERR_NULL), (dict(up_scales=None), qm.MOE_ERR_NULL), (dict(gate=A + 8), qm.MOE_ERR_ALIGN),
    (dict(down_scales=A + 1), qm.MOE_ERR_ALIGN), (dict(xq=A + 4), qm.MOE_ERR_ALIGN), (dict(n=4096), qm.MOE_ERR_WORKSPACE),
    (dict(wr=None, bias=A), qm.MOE_ERR_UNSUPPORTED),
])
def test_layer_refusals(over, code):
    assert layer(**over) == code


def test_layer_of_no_tokens():
    assert layer(s=shape(T=0), x=None, xq=None, out=None, ws=None, n=0, ex=False) == qm.MOE_OK


def test_python_takes_device_tensors_only():
    import torch
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    q, s = torch.zeros((4, 256), dtype=torch.uint8), torch.ones((4, 2))
    for call in (lambda: qm.add_rmsnorm(x), lambda: qm.gemm_fp8(q, s, q, torch.ones((1, 2))),
                 lambda: qm.grouped_gemm_fp8(q, s, q[None], s[None], torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError, match="device tensors"):
            call()
