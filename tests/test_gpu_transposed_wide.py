"""The transposed quantiser on matrices of few rows and very many columns."""
import pytest
import torch

import mxfp4_quantised_mixture_b200 as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [0, 1])
@pytest.mark.parametrize("cols", [1 << 27, (1 << 28) + 8])
def test_one_row_of_very_many_columns(cuda_device, cols, E):
    gen = torch.Generator(device=cuda_device).manual_seed(E)
    w = torch.randn((1, cols), generator=gen, device=cuda_device, dtype=torch.bfloat16)
    P = moe.mxfp4_transposed_width(1, E)
    q = torch.full((cols, P // 2), 0xAB, dtype=torch.uint8, device=cuda_device)
    s = torch.full((cols, P // 32), 0xAB, dtype=torch.uint8, device=cuda_device)
    if E:
        off = torch.tensor([0, 1], dtype=torch.int32, device=cuda_device)
        moe.mxfp4_quantize_transposed_grouped(w, off, q, s)
    else:
        moe.mxfp4_quantize_transposed(w, q, s)
    # the row quantiser on the transpose, padded to P: pieces from the start, the middle and the end
    n = 1 << 16
    for lo in (0, cols // 2 - 3, cols - n):
        t = torch.zeros((n, P), dtype=torch.bfloat16, device=cuda_device)
        t[:, 0] = w[0, lo:lo + n]
        rq, rs = torch.empty_like(q[:n]), torch.empty_like(s[:n])
        moe.mxfp4_quantize(t, rq, rs)
        assert torch.equal(q[lo:lo + n], rq) and torch.equal(s[lo:lo + n], rs)
    # everywhere else: 31 (127) of a column's positions hold the zero code, so behind the first byte
    # nothing is set
    assert not bool(q[:, 1:].any()) and not bool((q[:, 0] >> 4).any())
