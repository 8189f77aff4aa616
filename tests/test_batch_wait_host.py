"""moe_lora_add_polls on the host (no GPU needed): how often a workgroup may ask
is checked like every other argument, before any HIP call."""

import pytest

import quantized_routed_moe_amd as qm

A = 0x10000            # fake, 16-byte aligned "device" address (never dereferenced)


def add(polls, T=4, x=A):
    return qm.lib().moe_lora_add_polls(T, 64, 100, 16, 8, x, 64, A, A, A, A, A, A, 100, 2 * A, 100, qm.MOE_TYPE_BF16, A, 1 << 62,
                                       polls, None)


@pytest.mark.parametrize("polls", [-1, -(1 << 31), (1 << 18) + 1, (1 << 31) - 1])
def test_polls_outside_their_range(polls):
    assert add(polls) == qm.MOE_ERR_SHAPE
    assert add(polls, T=0) == qm.MOE_ERR_SHAPE


@pytest.mark.parametrize("polls", [0, 1, 1 << 14, 1 << 18])
def test_polls_within_it(polls):
    assert add(polls, T=0) == qm.MOE_OK
    assert add(polls, x=None) == qm.MOE_ERR_NULL
