"""moe_swiglu_quantize_e4m3: what a value becomes depends on its own gate and up
value and on its block's largest magnitude, and on nothing else."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,I", [(16384, 128), (4096, 640), (1001, 1152)])
@pytest.mark.parametrize("gate,up", [(-80.0, None), (float("nan"), None), (float("inf"), 1.0),
                                     (None, float("inf")), (3e38, 3e38), (-69.0, 2.0)])
def test_blocks_do_not_see_one_another(T, I, gate, up):
    """One far, infinite or NaN value in every third block: all the other blocks
    keep their bits. (A formula that differs by an ulp of fp32 for a neighbour's
    sake shows in one of some 2^18 codes, which is why there are millions.)"""
    import block_fp8_routed_amd as moe
    g = torch.Generator(device="cuda").manual_seed(T + I)
    gu = (torch.randn(T, 2 * I, generator=g, device="cuda") * 2.0).to(torch.bfloat16)
    codes, exps = moe.moe_swiglu_quantize_e4m3(gu)
    other = gu.clone()
    hit = torch.zeros(T * (I // 128), dtype=torch.bool, device="cuda")
    hit[::3] = True
    hit = hit.view(T, I // 128)
    where = torch.zeros(T, I // 128, 128, dtype=torch.bool, device="cuda")
    where[:, :, 37] = hit
    where = where.view(T, I)
    if gate is not None:
        other[:, :I] = torch.where(where, gate, other[:, :I])
    if up is not None:
        other[:, I:] = torch.where(where, up, other[:, I:])
    codes2, exps2 = moe.moe_swiglu_quantize_e4m3(other)
    torch.cuda.synchronize()
    assert torch.equal(exps2[~hit], exps[~hit])
    a, b = (c.view(T, I // 128, 128)[~hit] for c in (codes, codes2))
    assert torch.equal(a, b), f"{int((a != b).sum())} of {a.numel()} codes changed"


def test_far_values_leave_millions_of_neighbours_alone():
    """Every gate of magnitudes 2^-6 .. 69 beside random ups, 64 million values, a
    gate of -80 in every third block."""
    import block_fp8_routed_amd as moe
    T, I = 262144, 256
    g = torch.Generator(device="cuda").manual_seed(5)
    bits = torch.arange(0x3c80, 0x428a, device="cuda", dtype=torch.int32)
    bits = torch.cat([bits, bits + 0x8000]).to(torch.int16).view(torch.bfloat16)
    gu = torch.empty(T, 2 * I, dtype=torch.bfloat16, device="cuda")
    gu[:, :I] = bits[torch.randint(len(bits), (T, I), generator=g, device="cuda")]
    gu[:, I:] = torch.randn(T, I, generator=g, device="cuda").to(torch.bfloat16)
    gu[:, 7:I:128] = 0.0
    codes, exps = moe.moe_swiglu_quantize_e4m3(gu)
    hit = torch.zeros(T * 2, dtype=torch.bool, device="cuda")
    hit[::3] = True
    hit = hit.view(T, 2)
    gu[:, 7:I:128] = torch.where(hit, -80.0, 0.0).to(torch.bfloat16)
    codes2, exps2 = moe.moe_swiglu_quantize_e4m3(gu)
    torch.cuda.synchronize()
    assert torch.equal(exps2[~hit], exps[~hit])
    n = int((codes.view(T, 2, 128) != codes2.view(T, 2, 128))[~hit].sum())
    assert n == 0, f"{n} codes changed"


@pytest.mark.parametrize("gate", [-80.0, float("nan")])
def test_values_do_not_see_their_neighbours(gate):
    """Within a block whose largest magnitude stays, the other values keep
    their codes too (a gate of -80 gives 0, a NaN takes no part in the scale)."""
    import block_fp8_routed_amd as moe
    T, I = 16384, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    gu = (torch.randn(T, 2 * I, generator=g, device="cuda") * 2.0).to(torch.bfloat16)
    gu[:, 5], gu[:, I + 5] = 0.0, 0.0   # the value that changes is none of the largest
    codes, exps = moe.moe_swiglu_quantize_e4m3(gu)
    other = gu.clone()
    other[:, 5], other[:, I + 5] = gate, 1.0
    codes2, exps2 = moe.moe_swiglu_quantize_e4m3(other)
    torch.cuda.synchronize()
    assert torch.equal(exps2, exps)
    keep = torch.arange(I, device="cuda") != 5
    assert torch.equal(codes2[:, keep], codes[:, keep])
