"""Limits and refusals of the FP8 entry points that need no GPU."""

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
