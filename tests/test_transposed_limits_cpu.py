"""The size limits of the transposed quantiser, as the header states them
(nothing reaches a device here)."""
import pytest
import torch

import mxfp4_quantised_mixture_b200 as moe

L = moe.lib


def whole(batch, rows, cols):
    return L.mxfp4_quantize_transposed(16, batch, rows, cols, 16, 16, None, None)


def grouped(rows, cols, E):
    return L.mxfp4_quantize_transposed_grouped(16, rows, cols, 16, E, 16, 16, None, None)


def test_sizes_past_the_tile_limit_are_refused():
    # batch * ceil(P / 128) * ceil(cols / 128) past 2^31, while batch * rows * cols <= 2^40
    assert whole((1 << 31) + 1, 1, 8) == moe.MOE_ERR_SHAPE
    assert whole((1 << 30) + 1, 1, 136) == moe.MOE_ERR_SHAPE
    assert whole(129, 1, 1 << 31) == moe.MOE_ERR_SHAPE
    assert grouped(1, 1 << 31, 256) == moe.MOE_ERR_SHAPE  # 254 tiles of positions
    # no rows: nothing to do at any width
    assert grouped(0, 1 << 31, 256) == moe.MOE_OK and whole(1, 0, 1 << 31) == moe.MOE_OK


def test_sizes_up_to_the_tile_limit_are_taken():
    if torch.cuda.is_available():
        pytest.skip("its placeholder pointers must never reach a device")
    no_device = (moe.MOE_ERR_CUDA, moe.MOE_ERR_UNSUPPORTED)
    assert whole(1 << 31, 1, 8) in no_device and whole(128, 1, 1 << 31) in no_device
    assert whole(1, 1, 1 << 31) in no_device and whole(1, 512, 1 << 31) in no_device
    assert grouped(1, 1 << 31, 1) in no_device
