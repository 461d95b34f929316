"""Which kernel a 4-bit product takes (host only: the tiles of larger batches alone have a
workspace): the stream multiplies all columns that its wavefronts cover, so products of
few columns, or of a few more than one pass holds, go to the tiles at fewer rows than K
says. Sizes at which one of the two was measured at least 1.4 times as fast."""
import pytest

import block_fp8_routed_amd as moe

# rows, features, columns: stream us, tiles us (bf16 / fp32 output)
TILES = [(4096, 4096, 32),      # 92, 20 / 34
         (16384, 512, 32),      # 49, 21 / 24
         (1024, 4096, 64),      # 27, 14 / 17
         (8192, 1280, 64), (8192, 2048, 32),
         (4096, 1280, 128),     # 28, 15 / 16
         (4096, 4096, 256),     # 77, 26 / 38
         (1024, 4096, 1056),    # 56, 28 / 34
         (1024, 1280, 4128),    # 132, 68 / 60
         (256, 4096, 4128)]     # 103, 69 / 58
GROUPED_TILES = [(103, 222, 8026, 192, moe.MOE_F32),   # rows, experts, ...: 62, 34
                 (565, 38, 704, 4224, moe.MOE_F32)]    # 71, 43
STREAM = [(1, 4096, 32), (64, 512, 64), (1024, 512, 4096),  # 19, 47
          (256, 4096, 4096),    # 27, 44
          (64, 4096, 4128),     # 28, 69 / 56
          (256, 1280, 4128),    # 35, 64 / 55
          (1024, 1280, 4096),   # 33, 48
          (16, 8192, 8192)]


@pytest.mark.parametrize("dtype", [moe.MOE_BF16, moe.MOE_F32])
def test_products_take_the_faster_kernel(dtype):
    took = {size: moe.linear_w4_workspace_bytes(size[0], 1, *size[1:], dtype) > 0
            for size in TILES + STREAM}
    assert took == {size: size in TILES for size in TILES + STREAM}


def test_short_tiles_of_experts_count_in_full():
    """The stream takes 16 rows at a time, also for an expert that has one."""
    for *size, dtype in GROUPED_TILES:
        assert moe.linear_w4_workspace_bytes(*size, dtype) > 0, size
    # a decode batch's banks stay a stream of weights
    for size in ((80, 512, 2048, 4096), (128, 128, 1536, 2048), (128, 128, 2048, 768)):
        assert moe.linear_w4_workspace_bytes(*size, moe.MOE_BF16) == 0, size
