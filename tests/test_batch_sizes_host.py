"""Sizes of more than 32 bits through the Python entry points of a batch of many
requests (no GPU needed: tensors without memory, whose addresses the library
is not reached with): the C entry points take 32 bits, so what is left of such a
size could be a valid one."""

import pytest
import torch

import quantized_routed_moe_amd as qm

FAR = 1 << 32


def empty(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.fixture(autouse=True)
def no_device(monkeypatch):
    monkeypatch.setattr(qm, "_elsewhere", lambda dev, stream, where: None)
    monkeypatch.setattr(qm, "_raw_stream", lambda dev: None)


def a_plan(T, L):
    p = qm.LoraPlan.__new__(qm.LoraPlan)
    p.T, p.adapters, p.dev, p.perm_addr, p.items_addr = T, L, -1, None, None
    return p


def a_lora(T=4, K=64, N=40, r=8, L=3):
    return qm.lora_add(empty(T, N), empty(T, K), empty(L, r, K), empty(L, N, r), a_plan(T, L))


def a_row(V=100, T=1, given=1, **more):
    return qm.token_logprobs(empty(T, V), empty(T, given, dtype=torch.int32), **more)


@pytest.mark.parametrize("call", [
    lambda: qm.lora_plan(empty(FAR + 5, dtype=torch.int32), 3), lambda: qm.lora_plan(empty(5, dtype=torch.int32), FAR + 3),
    lambda: qm.lora_plan(empty(5, dtype=torch.int32), 3 - FAR),
    lambda: a_lora(T=FAR + 4), lambda: a_lora(K=FAR + 64), lambda: a_lora(N=FAR + 40), lambda: a_lora(r=FAR + 8), lambda: a_lora(L=FAR + 3),
    lambda: a_row(V=FAR + 100), lambda: a_row(T=FAR + 1), lambda: a_row(given=FAR + 1), lambda: a_row(top=FAR + 3),
], ids=["tokens", "adapters", "adapters below", "T", "K", "N", "r", "L", "V", "rows", "given", "top"])
def test_sizes_past_32_bits_are_refused(call):
    with pytest.raises(qm.MoeError) as e:
        call()
    assert e.value.code == qm.MOE_ERR_SHAPE


def test_sizes_of_32_bits_reach_the_library():
    """The same calls with sizes that fit get as far as their missing addresses."""
    for call in (lambda: qm.lora_plan(empty(5, dtype=torch.int32), 3), a_lora, a_row):
        with pytest.raises(qm.MoeError) as e:
            call()
        assert e.value.code == qm.MOE_ERR_NULL


def test_a_plan_of_sizes_past_32_bits_is_refused(monkeypatch):
    t = torch.empty(4, dtype=torch.int32)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    for T, L in ((FAR + 4, 3), (4, FAR + 3)):
        with pytest.raises(qm.MoeError) as e:
            qm.LoraPlan(T, L, t, t, t)
        assert e.value.code == qm.MOE_ERR_SHAPE
