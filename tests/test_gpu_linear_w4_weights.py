"""The weights of larger batches with bf16 output (tiles), which are rounded to fp16:
q - z is exact and the scale multiplies it, so that a weight is off by a part of itself.

The bound of an element. S, the scale times a power of two that brings the row's largest
to [2^14, 2^15), is rounded once to fp16's 11 bits, and so is the product S (q - z) 2^-9:
2^-11 of the weight each time, 2^-10 (1 + 2^-12) of it together. Below fp16's normal
numbers a rounding is off by up to 2^-25 instead; beside 2^14 2^-9, the smallest that the
largest scale is there, 2^-30 of that scale for the product, 2^-39 |q - z| of it for S.
fp32 sums as in test_gpu_linear_w4.py. A row of x is fp16 times the power of two that
brings its largest magnitude to 2^14 at least: half a step of fp16's smallest numbers,
2^-25, is up to 2^-39 of it.
The bound in norm. A rounding to 11 bits is off by 2^-11 / sqrt(3) of the value at most in
the mean square. Products round each for itself, S once a group: with codes drawn evenly
about the zero point the terms of a sum are as good as independent between columns and
between groups, so two such roundings leave sqrt(2 / 3) 2^-11 of the root of the sum of
their squares, counted here as 2^-11. The output's own rounding is that of the reference
(its norm is taken), independent of the weights'. 2% on top are for the sample: a row's
features, 1000 at least, each with errors of its own."""
import numpy as np
import pytest
import torch

from test_gpu_dispatch import HALF
from test_gpu_linear_w4 import takes_tiles, values

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def pack(q):
    return torch.from_numpy((q[..., 0::2] | q[..., 1::2] << 4).astype(np.uint8)).cuda()


def bound(x, w, s, z):
    """(result, bound of the error before its rounding, root of the sum of squares)."""
    x = x.double().cpu().numpy()
    v, mag, _ = values(w, s, z)
    a, top = np.abs(x), s.double().abs().amax(dim=1).cpu().numpy()
    err = ((64 + x.shape[1] / 32) * 2.0 ** -24 * (a @ mag.T)
           + 2.0 ** -39 * a.max(axis=1)[:, None] * np.abs(v).sum(axis=1)
           + 2.0 ** -10 * (1 + 2.0 ** -12) * (a @ np.abs(v).T)
           + (2.0 ** -30 + 255 * 2.0 ** -39) * a.sum(axis=1)[:, None] * top)
    return x @ v.T, err, np.sqrt((x * x) @ (v * v).T)


def check_tiles(got, x, w, s, z):
    y, err, square = bound(x, w, s, z)
    off = got.double().cpu().numpy() - y
    lim = err + HALF[BF16] * (np.abs(y) + err)
    assert (np.abs(off) <= lim).all(), f"{np.max(np.abs(off) / lim):.2f} of an element's bound"
    norm = np.linalg.norm
    own = norm(torch.from_numpy(y).to(BF16).double().numpy() - y)
    lim = 1.02 * np.hypot(own, 2.0 ** -11 * norm(square))
    assert norm(off) <= lim, f"{norm(off) / norm(y):.2e} in norm, bound {lim / norm(y):.2e}"


SIZES = [(2100, 1030, 1056, 32), (1800, 1280, 2176, 128), (1100, 2050, 1024, 64)]  # M, N, K, group


@pytest.mark.parametrize("M,N,K,G", SIZES)
@pytest.mark.parametrize("swiglu", [False, True])
def test_weights_at_their_zero_points_are_zero(M, N, K, G, swiglu):
    """q = z everywhere, scales of any value: the output is the bias, with SwiGLU 0 where
    a half of it is."""
    import block_fp8_routed_amd as moe
    assert takes_tiles(M, N, K, BF16)
    r = np.random.default_rng(M)
    z = r.integers(0, 16, (N, K // G)).astype(np.uint8)
    w = pack(np.repeat(z, G, axis=1))
    s = torch.from_numpy(np.exp(r.uniform(-6, 2, z.shape)).astype(np.float32)).cuda()
    x = torch.from_numpy((1 + 0.5 * r.normal(size=(M, K))).astype(np.float32)).to(BF16).cuda()
    bias = torch.from_numpy(r.normal(size=N).astype(np.float32)).cuda()
    zero = torch.from_numpy(z).cuda()
    assert bool((moe.moe_linear_w4(x, w, s, zero, swiglu=swiglu) == 0).all())
    if swiglu:
        bias[N // 4:N // 2], bias[N // 2:N * 3 // 4] = 0, 0
        assert bool((moe.moe_linear_w4(x, w, s, zero, bias=bias, swiglu=True) == 0).all())
    else:
        got = moe.moe_linear_w4(x, w, s, zero, bias=bias)
        assert torch.equal(got, bias.to(BF16).expand(M, N))
    half = M // 3
    offsets = torch.tensor([0, half, M - 5], dtype=torch.int32).cuda()
    out = torch.full((M, N // 2 if swiglu else N), 3.0, dtype=BF16, device="cuda")
    both = [torch.stack((t, t.flip(0))) for t in (w, s, zero)]
    moe.moe_grouped_linear_w4(x, offsets, *both, swiglu=swiglu, out=out)
    assert bool((out[:M - 5] == 0).all()) and bool((out[M - 5:] == 3).all())


@pytest.mark.parametrize("M,N,K,G", SIZES)
@pytest.mark.parametrize("zero", [7, 8, 9, 11])
@pytest.mark.parametrize("rows", ["about_0", "about_1", "near_1", "positive"])
def test_rows_with_a_mean(M, N, K, G, zero, rows):
    """Codes balanced about the zero point, rows whose values are not balanced about 0."""
    import block_fp8_routed_amd as moe
    assert takes_tiles(M, N, K, BF16)
    r = np.random.default_rng(M + zero)
    width = min(zero, 15 - zero)
    w = pack(r.integers(zero - width, zero + width + 1, (N, K)))
    s = (np.exp2(r.uniform(-1, 1, (N, K // G))) * 0.02).astype(np.float32)
    z = torch.full((N, K // G), zero, dtype=torch.uint8).cuda()
    n = r.normal(size=(M, K))
    x = {"about_0": n, "about_1": 1 + n, "near_1": 1 + 0.1 * n, "positive": np.abs(n)}[rows]
    x = torch.from_numpy(x.astype(np.float32)).to(BF16).cuda()
    for scales in (torch.from_numpy(s).cuda(), torch.from_numpy(s).to(BF16).cuda()):
        check_tiles(moe.moe_linear_w4(x, w, scales, z), x, w, scales, z)


@pytest.mark.parametrize("M,N,K,G", SIZES)
@pytest.mark.parametrize("b", [6, 10, 14, 20])
@pytest.mark.parametrize("zeros", [False, True])
def test_groups_of_small_scales_count(M, N, K, G, b, zeros):
    """One group's scales 2^b above the others', x as much larger where they are small:
    all groups bear alike on the result."""
    import block_fp8_routed_amd as moe
    assert takes_tiles(M, N, K, BF16)
    r = np.random.default_rng(M + b)
    zero = 9 if zeros else 8
    w = pack(r.integers(zero - 6, zero + 7, (N, K)))
    s = (np.exp2(r.uniform(-1, 1, (N, K // G))) * 0.02).astype(np.float32)
    x = r.normal(size=(M, K)) * 2.0 ** b
    s[:, 3] *= 2.0 ** b
    x[:, 3 * G:4 * G] *= 2.0 ** -b
    s = torch.from_numpy(s).cuda()
    z = torch.full(s.shape, zero, dtype=torch.uint8).cuda() if zeros else None
    x = torch.from_numpy(x.astype(np.float32)).to(BF16).cuda()
    check_tiles(moe.moe_linear_w4(x, w, s, z), x, w, s, z)
