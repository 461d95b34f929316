"""Dense block-FP8 products at the ends of their operands' ranges."""
import numpy as np
import pytest
import torch

from test_gpu_linear import compare, rows, run, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    import block_fp8_routed_amd as moe
    moe.load()
    yield
    torch.cuda.synchronize()


# one size for the stream that quantises, the stream on codes, and each fp32 tile
@pytest.mark.parametrize("M,N,out_dtype", [
    (2, 300, torch.float32), (2, 300, torch.bfloat16), (30, 300, torch.float32),
    (140, 5300, torch.bfloat16), (300, 4000, torch.float32), (700, 5000, torch.float32),
    (2200, 5000, torch.float32), (300, 4000, torch.bfloat16), (700, 5000, torch.bfloat16),
    (2200, 5000, torch.bfloat16)])
def test_smallest_activations_and_largest_scales(M, N, out_dtype):
    """bf16 values down to the smallest subnormal (exponents down to -127) with
    weight scales up to 2^99: every product's share is in the result, which is
    an ordinary number."""
    K = 512
    x = rows(M, K, M)
    x = (x.float() * 2.0 ** -116).to(torch.bfloat16)
    x[0] = (x[0].float() * 2.0 ** -8).to(torch.bfloat16)   # subnormal bf16 values
    x[1] = 2.0 ** -133
    x[M - 1, ::128] = 1.0                                  # an ordinary block beside them
    s = np.exp2(np.random.default_rng(M).uniform(90, 99.9, (-(-N // 128), K // 128)))
    y = run(M, N, K, out_dtype, x=x, scales=s.astype(np.float32))
    assert bool((y[1] != 0).any())


@pytest.mark.parametrize("M,N,out_dtype", [
    (2, 300, torch.float32), (30, 300, torch.bfloat16), (300, 4000, torch.float32),
    (2200, 5000, torch.float32), (300, 4000, torch.bfloat16), (700, 5000, torch.bfloat16),
    (2200, 5000, torch.bfloat16)])
def test_largest_sums(M, N, out_dtype):
    """Rows of the largest bf16 value, with the signs of a weight row of +-448,
    so that every product of a block adds up; and the same rows with the largest
    value of which the exponent below takes codes of 448."""
    K = 256
    g = np.random.default_rng(M)
    w, _ = weights(N, K, M)
    sign = np.where(g.random(K) < 0.5, -1.0, 1.0).astype(np.float32)
    w[5] = np.where(sign < 0, 0xFE, 0x7E)
    x = rows(M, K, M)
    x[0] = torch.from_numpy(sign).to(torch.bfloat16) * torch.finfo(torch.bfloat16).max
    x[1] = torch.from_numpy(sign * np.float32(448.0 * 2.0 ** 119)).to(torch.bfloat16)
    s = np.full((-(-N // 128), K // 128), 2.0 ** -40, np.float32)
    wd, sd = torch.from_numpy(w).cuda(), torch.from_numpy(s).cuda()
    import block_fp8_routed_amd as moe
    import oracle
    codes, exps = oracle.quantise_activations(x.float().numpy(), 128)
    assert exps[0, 0] == 120 and exps[1, 0] == 119
    y = moe.moe_linear(x.cuda(), wd, sd, out_dtype=out_dtype)
    compare(y, codes, exps, w, s, None, K, f"largest sums M={M} N={N} {out_dtype}")
