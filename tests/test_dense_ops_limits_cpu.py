"""Sizes at which the gated choice has to refuse a call on the host (no GPU): its
grid, four tokens a workgroup of 256, holds fewer than 2^32 threads."""
import ctypes

import pytest
import torch

import block_fp8_routed_amd as moe

P = 0x1000  # never dereferenced


@pytest.mark.parametrize("tokens", [(1 << 26) - 3, (1 << 26) - 1, 1 << 26, 1 << 40])
def test_choice_refuses_more_tokens_than_its_grid_holds(tokens):
    st = moe.load().moe_select_experts(P, moe.MOE_F32, 512, None, moe.Gating().ref, tokens, 512, 8,
                                       P, P, None)
    assert st == moe.MOE_ERR_UNSUPPORTED


def layer(tokens):
    """A small layer of many tokens, and workspace enough by its own account."""
    cfg = moe.make_config(tokens, 64, 8, 32, 2, 32, False, torch.float32)
    return cfg, moe.workspace_bytes(cfg)


@pytest.mark.parametrize("tokens", [(1 << 26) - 3, 1 << 26, 1 << 28])
def test_layer_with_the_choice_refuses_them_before_any_launch(tokens):
    cfg, n = layer(tokens)
    lib, g = moe.load(), moe.Gating()
    assert lib.moe_route_gated(P, P, None, None, g.ref, P, P, None, ctypes.byref(cfg), P, n,
                               None) == moe.MOE_ERR_UNSUPPORTED
    bank = moe.MoeExpertBank(P, P, P, P)
    assert lib.moe_forward_gated(P, P, None, None, g.ref, ctypes.byref(bank), None, 2, P,
                                 ctypes.byref(cfg), P, n, None, None) == moe.MOE_ERR_UNSUPPORTED
