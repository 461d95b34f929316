"""The current stream and device that the gated choice and the dense operators run
on, through torch's raw handles and through its public functions."""
import pytest
import torch

from test_gpu_gate_select import SIGMOID8, draw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("public", [False, True])
def test_current_stream_is_the_one_used(public, monkeypatch):
    import block_fp8_routed_amd as moe
    from block_fp8_routed_amd import _lib
    if public:
        monkeypatch.setattr(_lib, "_raw_stream", _lib._public_stream)
        monkeypatch.setattr(_lib, "_raw_device", torch.cuda.current_device)
    l = draw(2000, 256, 3).cuda()
    want = moe.moe_select_experts(l, 8, moe.Gating(**SIGMOID8))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert _lib._raw_stream(0) == torch.cuda.current_stream(0).cuda_stream
    with torch.cuda.stream(side):
        assert _lib._raw_stream(0) == side.cuda_stream
        # work that only the current stream's order puts after the copy
        moved = torch.zeros_like(l)
        for _ in range(20):
            moved.zero_()
        moved.copy_(l)
        got = moe.moe_select_experts(moved, 8, moe.Gating(**SIGMOID8))
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert _lib._raw_device() == torch.cuda.current_device()
