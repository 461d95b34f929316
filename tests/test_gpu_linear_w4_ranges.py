"""Products with 4-bit weights where the stream goes over K in several passes, by expert
and with SwiGLU, and with scales at the ends of their range. Bounds as derived in
test_gpu_linear_w4.py and, for the fp16 weights of larger batches with bf16 output, in
test_gpu_linear_w4_weights.py."""
import numpy as np
import pytest
import torch

from test_gpu_dispatch import TYPES
from test_gpu_linear_w4 import (activations, check, grouped_reference, reference, takes_tiles,
                                weights)
from test_gpu_linear_w4_weights import bound

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 5, 16, 33, 90])
@pytest.mark.parametrize("N,K,G", [(112, 8320, 64), (34, 4128, 32), (64, 12288, 128)])
def test_swiglu_of_several_passes(M, N, K, G):
    import block_fp8_routed_amd as moe
    w, s, z, b = weights((), N, K, G, M, "bf16", M % 2 == 1, True)
    s = s * 0.03  # (gates of about 1.5: the bound of the SwiGLU holds up to 8)
    x = activations(M, K, M)
    for out in TYPES.values():
        assert not takes_tiles(M, N, K, out)
        got = moe.moe_linear_w4(x, w, s, z, bias=b, swiglu=True, out_dtype=out)
        check(got, *reference(x, w, s, z, b, True, False), str(out))


@pytest.mark.parametrize("counts", [[3, 0, 17, 1, 40, 0], [0, 16, 0], [1] * 20, [0, 0, 35]])
@pytest.mark.parametrize("N,K,G", [(72, 8320, 64), (34, 4128, 32), (50, 4224, 128)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_experts_of_several_passes(counts, N, K, G, swiglu):
    import block_fp8_routed_amd as moe
    E, behind = len(counts), 5
    offsets = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    M = int(offsets[-1]) + behind
    w, s, z, b = weights((E,), N, K, G, 3, "f32", G != 64, True)
    s = s * 0.03
    x = activations(M, K, 4)
    ref, err = grouped_reference(x, offsets, w, s, z, b, swiglu, False)
    for kind in TYPES.values():
        assert not takes_tiles(M, N, K, kind, E)
        out = torch.full((M, N // 2 if swiglu else N), 6.0, dtype=kind, device="cuda")
        moe.moe_grouped_linear_w4(x, torch.from_numpy(offsets).cuda(), w, s, z, bias=b,
                                  swiglu=swiglu, out=out)
        check(out[:M - behind], ref[:M - behind], err[:M - behind], str(kind))
        assert bool((out[M - behind:] == 6).all())


# powers of two on scales (0.005 to 0.08 without) and activations (up to some 50)
@pytest.mark.parametrize("scale,row", [(93, -92), (93, 10), (-94, 96), (-94, 10), (-112, 111), (40, -118)])
@pytest.mark.parametrize("M,N,K,G", [(2, 40, 256, 128), (90, 40, 4224, 32), (4100, 900, 256, 64),
                                     (1100, 2050, 1056, 32)])
def test_scales_at_the_ends_of_their_range(M, N, K, G, scale, row):
    """The results are within fp32's range here; the scales and rows for themselves are far
    from 1, alone and together."""
    import block_fp8_routed_amd as moe
    w, s, z, _ = weights((), N, K, G, 10)
    s = s * 2.0 ** scale
    assert float(s.abs().max()) < 2.0 ** 90
    x = (activations(M, K, 11).float() * 2.0 ** row).to(torch.bfloat16)
    assert float(x.abs().max()) < 2.0 ** 120
    # (below 2^-126 fp32 keeps steps of 2^-149, one for each rounding of a sum of x q and of
    # what the scale makes of it)
    steps = 64 + K / 32
    tiny = steps * 2.0 ** -149 * (512 * float(s.abs().max()) * (K / G) * 20 + 512)
    for out in TYPES.values():
        if out == torch.bfloat16 and takes_tiles(M, N, K, out):
            ref, err, _ = bound(x, w, s, z)
        else:
            ref, err = reference(x, w, s, z, None, False, False)
        check(moe.moe_linear_w4(x, w, s, z, out_dtype=out), ref, err + tiny, str(out))


@pytest.mark.parametrize("M,N,K,G", [(4096, 4096, 32, 32), (4100, 1290, 64, 64), (4100, 1290, 64, 32),
                                     (4097, 1300, 128, 128), (3000, 2050, 96, 32), (4100, 1284, 192, 64),
                                     (1030, 1282, 4128, 32), (260, 4100, 4160, 64)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_few_columns_and_a_few_past_a_pass_on_tiles(M, N, K, G, swiglu):
    import block_fp8_routed_amd as moe
    for i, out in enumerate(TYPES.values()):
        assert takes_tiles(M, N, K, out)
        w, s, z, b = weights((), N, K, G, M + i, "bf16" if i else "f32", i == 0, True)
        s = s * (0.03 if swiglu else 1)
        x = activations(M, K, M)
        got = moe.moe_linear_w4(x, w, s, z, bias=b, swiglu=swiglu, out_dtype=out)
        if out == torch.bfloat16 and not swiglu:
            y, err, _ = bound(x, w, s, z)
            b = b.double().cpu().numpy()
            ref, err = y + b, err + 2.0 ** -24 * (np.abs(y) + np.abs(b))
        else:
            ref, err = reference(x, w, s, z, b, swiglu, out == torch.bfloat16)
        check(got, ref, err, str(out))


@pytest.mark.parametrize("M,E,N,K,G", [(103, 222, 8026, 192, 64), (565, 38, 704, 4224, 128)])
def test_short_tiles_of_experts(M, E, N, K, G):
    import block_fp8_routed_amd as moe
    assert takes_tiles(M, N, K, torch.float32, E)
    r = np.random.default_rng(M)
    offsets = np.searchsorted(np.sort(r.integers(0, E, M)), np.arange(E + 1)).astype(np.int32)
    w, s, z, b = weights((E,), N, K, G, 5, bias=True)
    x = activations(M, K, 6)
    got = moe.moe_grouped_linear_w4(x, torch.from_numpy(offsets).cuda(), w, s, z, bias=b,
                                    out_dtype=torch.float32)
    check(got, *grouped_reference(x, offsets, w, s, z, b, False, False))
