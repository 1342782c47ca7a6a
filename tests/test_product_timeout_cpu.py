"""mxfp4_matmul_ex takes and refuses what mxfp4_matmul does (nothing reaches a
device here)."""
import pytest
import torch

import mxfp4_quantised_mixture_b200 as moe

L = moe.lib


def call(a=16, sa=16, b=16, sb=16, M=4, N=8, K=64, out=16, kind=0, st=None, fail=0):
    return L.mxfp4_matmul_ex(a, sa, b, sb, M, N, K, 1.0, out, kind, st, fail, None)


def test_refusals():
    assert call(K=48) == moe.MOE_ERR_SHAPE and call(M=-1) == moe.MOE_ERR_SHAPE
    assert call(N=(1 << 27) + 1) == moe.MOE_ERR_SHAPE
    assert call(M=0) == moe.MOE_OK and call(N=0) == moe.MOE_OK
    assert call(a=None) == moe.MOE_ERR_INVALID_ARG and call(out=8) == moe.MOE_ERR_INVALID_ARG
    assert call(kind=2) == moe.MOE_ERR_INVALID_ARG and call(st=18) == moe.MOE_ERR_INVALID_ARG


def test_binding_refuses_what_does_not_belong_together():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    with pytest.raises(ValueError, match="mxfp4_matmul_ex: .* belong together"):
        moe.mxfp4_matmul_ex(u8(4, 32), u8(4, 2), u8(8, 16), u8(8, 2), torch.zeros((4, 8)))
    with pytest.raises(ValueError, match="CUDA device"):
        moe.mxfp4_matmul_ex(u8(4, 32), u8(4, 2), u8(8, 32), u8(8, 2), torch.zeros((4, 8)))
