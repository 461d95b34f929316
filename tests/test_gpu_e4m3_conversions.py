"""The conversion to E4M3 bytes that the activation quantiser and the SwiGLU make
with gfx950's scaled instructions, against the oracle's rounding: every bf16
value under every exponent that its block can have, and fp32 values sampled."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

BF16_MAX = float(torch.finfo(torch.bfloat16).max)


def bf16_values():
    """All finite bf16 values, as fp32 numbers, by magnitude."""
    b = np.arange(0x7F80, dtype=np.uint32)
    v = (np.concatenate([b, b | 0x8000]) << 16).view(np.float32)
    return v[np.argsort(np.abs(v), kind="stable")]


@pytest.mark.parametrize("low", range(-127, 121, 31))
def test_every_bf16_value_under_every_exponent(low):
    """A block's largest value sets its exponent e: 448 2^e (of bf16's end, where
    that is smaller), and beside it the values up to it, 127 to a block."""
    import block_fp8_routed_amd as moe
    values = bf16_values()
    for e in range(low, min(low + 31, 121)):
        top = np.float32(min(448.0 * 2.0 ** e, BF16_MAX))
        v = values[np.abs(values) <= top]
        # what lies 2^-30 below the largest is code 0 everywhere: a sample of it
        far = np.abs(v) < top * np.float32(2.0 ** -30)
        v = np.concatenate([v[far][::101], v[~far]])
        n = -(-len(v) // 127)
        x = np.zeros((n, 128), np.float32)
        x[:, 0] = top
        flat = np.zeros(n * 127, np.float32)
        flat[:len(v)] = v
        x[:, 1:] = flat.reshape(n, 127)
        want, exps = oracle.quantise_activations(x, 128)
        assert (exps == e).all()
        xd = torch.from_numpy(x).to(torch.bfloat16)
        assert torch.equal(xd.float(), torch.from_numpy(x))
        codes, got = moe.moe_quantize_act_e4m3(xd.cuda())
        assert (got.cpu().numpy().astype(np.int64) - 127 == e).all()
        bad = np.argwhere(codes.cpu().numpy() != want)
        assert not len(bad), f"e={e}: {len(bad)} codes, first {x[tuple(bad[0])]}"


@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** -20, 1.0, 2.0 ** 30, 2.0 ** 110])
def test_fp32_values(scale):
    """Through the SwiGLU: a gate of 96 or more is its own silu (e^-96 is lost
    beside 1), so h is the product of two bf16 values, exact in fp32."""
    import block_fp8_routed_amd as moe
    rng = np.random.default_rng(int(np.log2(scale)) + 200)
    T, I = 512, 1024
    g = torch.from_numpy(rng.uniform(96, 250, (T, I))).to(torch.bfloat16)
    u = torch.from_numpy(rng.standard_normal((T, I)) * scale
                         * np.exp2(rng.integers(-12, 3, (T, I)))).to(torch.bfloat16)
    # products that sit on midpoints between two codes, and next to them
    g[::2, 3:] = 128.0
    mid = 1.0 + (2 * rng.integers(0, 8, (T // 2, I - 3)) + 1) / 16.0
    u[::2, 3:] = torch.from_numpy(mid * scale * np.exp2(rng.integers(-9, 1, mid.shape))).to(torch.bfloat16)
    h = g.double().numpy() * u.double().numpy()
    assert np.array_equal(h, h.astype(np.float32))
    want, exps = oracle.quantise_activations(h, 128)
    codes, got = moe.moe_swiglu_quantize_e4m3(torch.cat([g, u], 1).cuda())
    assert np.array_equal(got.cpu().numpy().astype(np.int64) - 127, exps)
    assert np.array_equal(codes.cpu().numpy(), want)
