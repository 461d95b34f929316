"""Refusals of the gated choice and the dense operators on the host (no GPU):
every invalid call returns its status before any HIP call, and the Python
functions refuse what the C functions cannot see."""
import ctypes

import pytest
import torch

import block_fp8_routed_amd as moe
from block_fp8_routed_amd import _lib

P = 0x1000  # never dereferenced: validation fails, or there is nothing to do


def select(gating=None, dtype=0, ld=64, tokens=4, experts=64, top_k=4, logits=P, idx=P, gates=P,
           null_gating=False, **rule):
    g = gating or moe.Gating(**rule)
    return moe.load().moe_select_experts(logits, dtype, ld, None, None if null_gating else g.ref,
                                         tokens, experts, top_k, idx, gates, None)


def raw(**kw):
    base = dict(score=0, groups=1, top_groups=1, group_rank=1, renormalise=1, scale=1.0)
    base.update(kw)
    g = moe.Gating()
    g.c = _lib.MoeGating(*base.values())
    g.ref = ctypes.byref(g.c)
    return g


def test_select_accepts_no_tokens():
    assert select(tokens=0) == moe.MOE_OK
    assert select(tokens=0, groups=8, top_groups=2, group_rank=2) == moe.MOE_OK


@pytest.mark.parametrize("kw,status", [
    (dict(top_k=0), moe.MOE_ERR_SHAPE),
    (dict(top_k=65), moe.MOE_ERR_SHAPE),
    (dict(experts=0), moe.MOE_ERR_SHAPE),
    (dict(tokens=-1), moe.MOE_ERR_SHAPE),
    (dict(ld=63), moe.MOE_ERR_SHAPE),
    (dict(dtype=2), moe.MOE_ERR_SHAPE),
    (dict(dtype=-1), moe.MOE_ERR_SHAPE),
    (dict(top_k=17), moe.MOE_ERR_UNSUPPORTED),
    (dict(experts=1025, ld=2000), moe.MOE_ERR_UNSUPPORTED),
    (dict(tokens=1 << 32), moe.MOE_ERR_UNSUPPORTED),
    (dict(logits=None), moe.MOE_ERR_NULL),
    (dict(idx=None), moe.MOE_ERR_NULL),
    (dict(gates=None), moe.MOE_ERR_NULL),
    (dict(null_gating=True), moe.MOE_ERR_NULL),
    (dict(groups=0), moe.MOE_ERR_SHAPE),
    (dict(groups=3), moe.MOE_ERR_SHAPE),                    # does not divide the experts
    (dict(groups=8, top_groups=9), moe.MOE_ERR_SHAPE),
    (dict(groups=8, top_groups=0), moe.MOE_ERR_SHAPE),
    (dict(groups=32, top_groups=1), moe.MOE_ERR_SHAPE),     # two experts cannot give four
    (dict(groups=64, top_groups=8, group_rank=2), moe.MOE_ERR_SHAPE),
    (dict(group_rank=0), moe.MOE_ERR_SHAPE),
    (dict(group_rank=3), moe.MOE_ERR_SHAPE),
    (dict(scale=float("nan")), moe.MOE_ERR_SHAPE),
    (dict(scale=float("inf")), moe.MOE_ERR_SHAPE),
    (dict(experts=256, ld=256, groups=128, top_groups=64), moe.MOE_ERR_UNSUPPORTED),
])
def test_select_refusals(kw, status):
    assert select(**kw) == status


def test_grids_are_bounded():
    """Calls whose grid would pass 2^32 threads are refused, not launched."""
    assert select(tokens=1 << 26) == moe.MOE_ERR_UNSUPPORTED
    assert linear(rows=1 << 20, n=1 << 18, k=128, ld_out=1 << 18,
                  work_bytes=1 << 40) == moe.MOE_ERR_UNSUPPORTED


def test_select_refuses_bad_enums():
    assert select(gating=raw(score=2)) == moe.MOE_ERR_SHAPE
    assert select(gating=raw(score=-1)) == moe.MOE_ERR_SHAPE
    assert select(gating=raw(renormalise=2)) == moe.MOE_ERR_SHAPE
    with pytest.raises(ValueError):
        moe.Gating(score="tanh")


def layer_cfg(path="auto", **kw):
    base = dict(tokens=4, hidden=64, experts=8, inter=32, top_k=2, block=32,
                x_dtype=torch.float32, path=path)
    base.update(kw)
    return moe.make_config(**base)


def forward(cfg, gating, ws_bytes=None, x=P, top_k=None):
    b = _lib.MoeExpertBank(0x2000, 0x2000, 0x2000, 0x2000)
    n = moe.workspace_bytes(cfg) if ws_bytes is None else ws_bytes
    return moe.load().moe_forward_gated(x, P, None, None, gating.ref if gating else None,
                                        ctypes.byref(b), None, cfg.top_k if top_k is None else top_k,
                                        P, ctypes.byref(cfg), P, n, None, None)


def test_forward_gated_refusals():
    g = moe.Gating()
    assert forward(layer_cfg(), None) == moe.MOE_ERR_NULL
    assert forward(layer_cfg(), moe.Gating(groups=3)) == moe.MOE_ERR_SHAPE
    assert forward(layer_cfg(), moe.Gating(groups=8, top_groups=1)) == moe.MOE_ERR_SHAPE
    assert forward(layer_cfg("gemv_fused"), g) == moe.MOE_ERR_UNSUPPORTED
    assert forward(layer_cfg(), g, ws_bytes=16) == moe.MOE_ERR_WORKSPACE
    assert forward(layer_cfg(), g, x=None) == moe.MOE_ERR_NULL
    assert forward(layer_cfg(), g, top_k=3) == moe.MOE_ERR_SHAPE
    assert forward(layer_cfg(hidden=128, inter=64), g) == moe.MOE_ERR_UNSUPPORTED
    assert forward(layer_cfg(tokens=0), g) == moe.MOE_OK


def test_route_gated_refusals():
    c = layer_cfg()
    lib, ref = moe.load(), ctypes.byref(c)
    n = moe.workspace_bytes(c)
    g = moe.Gating()
    args = lambda **k: [k.get("x", P), P, None, None, k.get("g", g.ref), k.get("idx", P),  # noqa: E731
                        k.get("gates", P), None, ref, k.get("ws", P), k.get("n", n), None]
    assert lib.moe_route_gated(*args(g=None)) == moe.MOE_ERR_NULL
    assert lib.moe_route_gated(*args(x=None)) == moe.MOE_ERR_NULL
    assert lib.moe_route_gated(*args(idx=None)) == moe.MOE_ERR_NULL
    assert lib.moe_route_gated(*args(ws=None)) == moe.MOE_ERR_NULL
    assert lib.moe_route_gated(*args(n=8)) == moe.MOE_ERR_WORKSPACE
    assert lib.moe_route_gated(*args(ws=0x1010)) == moe.MOE_ERR_WORKSPACE
    assert lib.moe_route_gated(*args(g=moe.Gating(groups=5).ref)) == moe.MOE_ERR_SHAPE


def linear(x=P, ld_x=256, w=P, ws=P, rows=4, n=96, k=256, out=P, ld_out=96, dtype=0, work=P,
           work_bytes=1 << 30):
    return moe.load().moe_linear(x, ld_x, w, ws, None, rows, n, k, out, ld_out, dtype, work,
                                 work_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), moe.MOE_ERR_NULL),
    (dict(w=None), moe.MOE_ERR_NULL),
    (dict(ws=None), moe.MOE_ERR_NULL),
    (dict(out=None), moe.MOE_ERR_NULL),
    (dict(rows=-1), moe.MOE_ERR_SHAPE),
    (dict(n=0), moe.MOE_ERR_SHAPE),
    (dict(k=0), moe.MOE_ERR_SHAPE),
    (dict(k=-128), moe.MOE_ERR_SHAPE),
    (dict(ld_x=128), moe.MOE_ERR_SHAPE),
    (dict(ld_out=95), moe.MOE_ERR_SHAPE),
    (dict(dtype=2), moe.MOE_ERR_SHAPE),
    (dict(k=192), moe.MOE_ERR_UNSUPPORTED),
    (dict(ld_x=260), moe.MOE_ERR_UNSUPPORTED),     # rows not 16-byte aligned
    (dict(x=0x1008), moe.MOE_ERR_UNSUPPORTED),
    (dict(w=0x1004), moe.MOE_ERR_UNSUPPORTED),
    (dict(rows=1 << 21), moe.MOE_ERR_UNSUPPORTED),
    (dict(rows=0), moe.MOE_OK),
])
def test_linear_refusals(kw, status):
    assert linear(**kw) == status


def test_linear_workspace_refusals():
    n = moe.linear_workspace_bytes(500, 96, 256, False)
    assert n > 0
    assert linear(rows=500, work=None, work_bytes=0) == moe.MOE_ERR_NULL
    assert linear(rows=500, work_bytes=n - 1) == moe.MOE_ERR_WORKSPACE
    assert linear(rows=500, work=0x1010, work_bytes=n) == moe.MOE_ERR_WORKSPACE
    assert moe.linear_workspace_bytes(0, 96, 256, False) == 0
    assert moe.linear_workspace_bytes(4, 96, 200, False) == 0
    assert moe.linear_workspace_bytes(-4, 96, 256, True) == 0


def test_linear_e4m3_refusals():
    f = moe.load().moe_linear_e4m3
    ok = [P, P, P, P, None, 0, 96, 256, P, 96, 0, P, 1 << 30, None]
    assert f(*ok) == moe.MOE_OK  # no rows
    for at in (0, 1, 2, 3, 8):
        assert f(*[None if i == at else a for i, a in enumerate(ok)]) == moe.MOE_ERR_NULL
    assert f(0x1008, *ok[1:5], 4, *ok[6:]) == moe.MOE_ERR_UNSUPPORTED
    assert f(*ok[:7], 130, *ok[8:]) == moe.MOE_ERR_UNSUPPORTED


def test_swiglu_refusals():
    f = moe.load().moe_swiglu_quantize_e4m3
    assert f(P, 512, 0, 256, P, P, None) == moe.MOE_OK
    assert f(None, 512, 4, 256, P, P, None) == moe.MOE_ERR_NULL
    assert f(P, 512, 4, 256, None, P, None) == moe.MOE_ERR_NULL
    assert f(P, 512, 4, 256, P, None, None) == moe.MOE_ERR_NULL
    assert f(P, 511, 4, 256, P, P, None) == moe.MOE_ERR_SHAPE
    assert f(P, 512, -1, 256, P, P, None) == moe.MOE_ERR_SHAPE
    assert f(P, 512, 4, 0, P, P, None) == moe.MOE_ERR_SHAPE
    assert f(P, 512, 4, 192, P, P, None) == moe.MOE_ERR_UNSUPPORTED
    assert f(P, 516, 4, 256, P, P, None) == moe.MOE_ERR_UNSUPPORTED
    assert f(0x1008, 512, 4, 256, P, P, None) == moe.MOE_ERR_UNSUPPORTED
    assert f(P, 512, 4, 256, 0x1004, P, None) == moe.MOE_ERR_UNSUPPORTED
    assert f(P, 512, 1 << 40, 256, P, P, None) == moe.MOE_ERR_UNSUPPORTED


def test_python_refuses_host_tensors_and_wrong_types():
    cpu = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        moe.moe_select_experts(cpu, 2, moe.Gating())
    with pytest.raises(ValueError):
        moe.moe_linear(torch.zeros(2, 128, dtype=torch.bfloat16),
                       torch.zeros(8, 128, dtype=torch.uint8), torch.zeros(1, 1))
    with pytest.raises(ValueError):
        moe.moe_swiglu_quantize_e4m3(torch.zeros(2, 256, dtype=torch.bfloat16))
