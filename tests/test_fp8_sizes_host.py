"""Sizes of more than 32 bits through the Python entry points of the FP8 operators
(no GPU needed: tensors without memory): the C entry points take 32 bits, so what
is left of such a size could be a valid one."""

import pytest
import torch

import quantized_routed_moe_amd as qm

FAR = 1 << 32
F32, F8, BF16, I32 = torch.float32, torch.float8_e4m3fn, torch.bfloat16, torch.int32


def empty(*shape, dtype=F8):
    return torch.empty(shape, dtype=dtype, device="meta")


def runs(n):
    return (n + 127) // 128


@pytest.fixture(autouse=True)
def no_device(monkeypatch):
    monkeypatch.setattr(qm, "_elsewhere", lambda dev, stream, where: None)
    monkeypatch.setattr(qm, "_raw_stream", lambda dev: None)
    monkeypatch.setattr(qm, "_ptr", lambda t, *a, **k: None)
    monkeypatch.setattr(qm, "alloc_workspace_fp8", lambda *a, **k: empty(4096, dtype=torch.uint8))


def norm(T=4, d=256):
    return qm.add_rmsnorm(empty(T, d, dtype=BF16))


def gemm(M=4, N=256, K=128):
    return qm.gemm_fp8(empty(M, K), empty(M, runs(K), dtype=F32), empty(N, K), empty(runs(N), runs(K), dtype=F32))


def grouped(R=4, E=2, N=256, K=128, k=1, rows=None):
    return qm.grouped_gemm_fp8(empty(R, K), empty(R, runs(K), dtype=F32), empty(E, N, K), empty(E, runs(N), runs(K), dtype=F32),
                               empty(E + 1, dtype=I32), perm=None if rows is None else empty(rows, dtype=I32), k=k)


def gate_up(T=4, d=256, E=2, k=2, f=128):
    w, s = empty(E, f, d), empty(E, runs(f), runs(d), dtype=F32)
    return qm.expert_gate_up_fp8(empty(T, d), empty(T, runs(d), dtype=F32), w, s, w, s, empty(E + 1, dtype=I32), empty(T * k, dtype=I32), k)


def layer(T=4, d=256, E=2, k=2, f=128):
    w, s = empty(E, f, d), empty(E, runs(f), runs(d), dtype=F32)
    ex = qm.ExpertsFp8(w, s, w, s, empty(E, d, f), empty(E, runs(d), runs(f), dtype=F32))
    return qm.layer_fp8(None, empty(T, d), empty(T, runs(d), dtype=F32), ex, k, logits=empty(T, E, dtype=F32))


CALLS = dict(norm=(norm, "T d"), gemm=(gemm, "M N K"), grouped=(grouped, "R E N K k"), gate_up=(gate_up, "T d E k f"),
             layer=(layer, "T d E k f"))
LEFT = dict(T=4, d=256, M=4, N=256, K=128, R=4, E=2, k=2, f=128)


@pytest.mark.parametrize("name,size", [(n, s) for n, (_, sizes) in CALLS.items() for s in sizes.split()])
def test_sizes_past_32_bits_are_refused(name, size):
    with pytest.raises(qm.MoeError) as e:
        CALLS[name][0](**{size: FAR + LEFT[size]})
    assert e.value.code == qm.MOE_ERR_SHAPE


def test_rows_past_32_bits_are_refused():
    with pytest.raises(qm.MoeError) as e:
        grouped(rows=FAR + 4)
    assert e.value.code == qm.MOE_ERR_SHAPE


@pytest.mark.parametrize("name", list(CALLS))
def test_sizes_of_32_bits_reach_the_library(name):
    """The same calls with sizes that fit get as far as their missing addresses."""
    with pytest.raises(qm.MoeError) as e:
        CALLS[name][0]()
    assert e.value.code == qm.MOE_ERR_NULL
