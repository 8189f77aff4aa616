"""Limits and refusals of the FP8 entry points that need no GPU."""

import ctypes

import pytest
import torch

import quantized_routed_moe_amd as qm


def test_layer_needs_a_router_or_logits():
    """Without w_router the logits are an input; none given must not become
    uninitialised memory."""
    q, s = torch.zeros((4, 256), dtype=torch.uint8), torch.ones((4, 2))
    w, ws = torch.zeros((2, 128, 256), dtype=torch.uint8), torch.ones((2, 1, 2))
    d, ds = torch.zeros((2, 256, 128), dtype=torch.uint8), torch.ones((2, 2, 1))
    with pytest.raises(ValueError, match="w_router or logits"):
        qm.layer_fp8(None, q, s, qm.ExpertsFp8(w, ws, w, ws, d, ds), 1)


def test_workspace_is_a_device_tensor():
    with pytest.raises(ValueError, match="type cuda"):
        qm.alloc_workspace_fp8(qm.Shape(4, 256, 8, 2, 128), device="cpu")


A = 0x10000            # fake, 16-byte aligned "device" address (never dereferenced)


# A grid has fewer than 2^32 threads, which is 2^23 workgroups of 512, not the
# 2^31 of a workgroup's index: refused before any HIP call.

@pytest.mark.parametrize("M,N", [((1 << 30) - 1, 1), (1 << 20, 1 << 20), (129, (1 << 30) - 1), (1 << 29, 257)])
def test_gemm_of_more_tiles_than_a_grid_holds(M, N):
    assert qm.lib().moe_gemm_fp8(M, N, 32, A, 32, A, A, A, A, qm.MOE_TYPE_BF16, N, None) == qm.MOE_ERR_SHAPE


@pytest.mark.parametrize("R,N", [(128, (1 << 30) - 1), ((1 << 30) - 1, 1 << 12), (3, (1 << 30) - 1), (64, 1 << 25)])
def test_grouped_gemm_of_more_tiles_than_a_grid_holds(R, N):
    assert qm.lib().moe_grouped_gemm_fp8(R, 64, N, 32, A, R, A, A, A, A, None, 1, A, qm.MOE_TYPE_F32,
                                         None) == qm.MOE_ERR_SHAPE


def test_gate_up_of_more_tiles_than_a_grid_holds():
    s = ctypes.byref(qm.moe_shape(64, 32, 64, 2, (1 << 24) - 32))
    assert qm.lib().moe_expert_gate_up_fp8(s, A, A, A, A, A, A, A, A, A, A, A, 1 << 40, None) == qm.MOE_ERR_SHAPE
