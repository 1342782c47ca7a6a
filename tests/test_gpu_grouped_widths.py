"""Experts' products around the changes of tile width: even and crowded batches
whose mean rows per expert are 16 to 65."""
import pytest
import torch

import mxfp4_quantised_mixture_b200 as moe
from mx_plain import behind_untouched, guarded, product_bound, random_mx, value

pytestmark = pytest.mark.gpu


def even(E, per):
    return [per] * E


def crowded(E, per):
    """One expert has half of the rows, one none."""
    rest = (per // 2) * (E - 2)
    return [per * E - rest, 0] + [per // 2] * (E - 2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts_of", [even, crowded])
@pytest.mark.parametrize("E,per,N,K", [(6, 16, 200, 160), (6, 17, 2050, 288), (5, 33, 1301, 1056),
                                       (9, 48, 900, 2880), (4, 64, 384, 96), (7, 65, 130, 4128)])
def test_grouped_around_the_widths(cuda_device, E, per, N, K, counts_of, dtype):
    counts = counts_of(E, per)
    S = sum(counts)
    gen = torch.Generator(device=cuda_device).manual_seed(S + N + K)
    a, b = random_mx(gen, (S, K)), random_mx(gen, (E, N, K))
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32).to(cuda_device)
    out, whole = guarded((S, N), dtype, cuda_device, 77.0)
    st = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    moe.mxfp4_matmul_grouped(*a, off, *b, out, d_status=st)
    assert int(st) == 0
    av, lo = value(*a), 0
    for e, c in enumerate(counts):
        rows, be = av[lo:lo + c], value(b[0][e], b[1][e])
        want = rows @ be.T
        bound = product_bound(rows.abs() @ be.abs().T, K, 1.0, dtype, want)
        assert bool(((out[lo:lo + c].double() - want).abs() <= bound).all())
        lo += c
    assert behind_untouched(out, whole, 77.0)
