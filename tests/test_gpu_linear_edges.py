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


@pytest.mark.parametrize("M,N,K", [(2, 300, 512), (16, 8192, 4096), (30, 300, 512), (140, 5300, 512),
                                   (300, 4000, 512), (700, 5000, 512), (2200, 5000, 512)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_a_nan_code_makes_its_row_nan_and_no_other(M, N, K, out_dtype):
    """What moe_swiglu_quantize_e4m3 writes for a NaN h (a padding row, say)."""
    import block_fp8_routed_amd as moe
    w, s = (torch.from_numpy(a).cuda() for a in weights(N, K, M))
    codes, exps = moe.moe_quantize_act_e4m3(rows(M, K, M).cuda())
    want = moe.moe_linear_e4m3(codes, exps, w, s, out_dtype=out_dtype)
    for row, col, nan in ((0, 0, 0x7F), (M - 1, K - 1, 0x7F), (M // 2, 129, 0xFF)):
        bad = codes.clone()
        bad[row, col] = nan
        got = moe.moe_linear_e4m3(bad, exps, w, s, out_dtype=out_dtype)
        assert bool(got[row].isnan().all())
        keep = torch.arange(M, device="cuda") != row
        assert torch.equal(got[keep], want[keep])


def norm_of_rounding(y):
    """What rounding y to bf16 amounts to, of y, in norm."""
    r = torch.from_numpy(y).to(torch.bfloat16).double().numpy()
    return float(np.linalg.norm(r - y) / np.linalg.norm(y))


@pytest.mark.parametrize("M,N,K", [(300, 4000, 512), (700, 5000, 1024), (2200, 5000, 512)])
def test_cuts_of_the_fp8_instruction_in_norm(M, N, K):
    """Tile-sized products with bf16 output, against the rounding of their exact
    values. The instruction cuts each of eight products towards zero at 2^-13 of
    the largest one, p: a mean square of at most p^2 2^-26 / 3 each, of random
    sign, so 8/3 2^-26 of the squares' sum, which is the result's own expected
    square for terms of random sign: 2^-12.3 in norm. It joins the output's
    rounding in square. Twice the cuts are allowed for (the result's square is
    near its expectation, not on it)."""
    import block_fp8_routed_amd as moe
    import oracle
    x, (w, s) = rows(M, K, M), weights(N, K, M)
    codes, exps = oracle.quantise_activations(x.float().numpy(), 128)
    want, _ = oracle.linear_e4m3(codes, exps, w, s, None)
    y = moe.moe_linear(x.cuda(), torch.from_numpy(w).cuda(), torch.from_numpy(s).cuda())
    norm = float(np.linalg.norm(y.double().cpu().numpy() - want) / np.linalg.norm(want))
    rounding = norm_of_rounding(want)
    cut = (8 / 3) ** 0.5 * 2.0 ** -13
    print(f"norm {norm:.3e}, rounding {rounding:.3e}, cuts {max(norm ** 2 - rounding ** 2, 0) ** 0.5:.2e}")
    assert norm <= (rounding ** 2 + (2 * cut) ** 2) ** 0.5


@pytest.mark.parametrize("M,N,K", [(2, 300, 512), (16, 8192, 4096), (30, 300, 512), (77, 2112, 4096),
                                   (300, 4000, 512), (700, 5000, 512), (2200, 5000, 512)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_rows_beside_rows_that_are_not_finite(M, N, K, out_dtype):
    """Rows of padding that hold NaN or infinities are no supported input, and
    leave the others as they are."""
    import block_fp8_routed_amd as moe
    w, s = (torch.from_numpy(a).cuda() for a in weights(N, K, M))
    x = rows(M, K, M).cuda()
    want = moe.moe_linear(x, w, s, out_dtype=out_dtype)
    for row, value in ((0, float("nan")), (M - 1, float("inf")), (M // 2, float("-inf"))):
        bad = x.clone()
        bad[row, ::3] = value
        got = moe.moe_linear(bad, w, s, out_dtype=out_dtype)
        keep = torch.arange(M, device="cuda") != row
        assert torch.equal(got[keep], want[keep])
