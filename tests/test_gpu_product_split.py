"""When a product's few tiles share their contraction between the CTAs of a
cluster, seen by the number of CTAs launched: mxfp4_matmul_ex reports a timeout
for a CTA that exists, and runs normally for one that does not."""
import pytest
import torch

import mxfp4_quantised_mixture_b200 as moe
from mx_plain import product_bound, random_mx, value

pytestmark = pytest.mark.gpu


def run(dev, M, N, K, cta):
    gen = torch.Generator(device=dev).manual_seed(M + N + K)
    a, b = random_mx(gen, (M, K)), random_mx(gen, (N, K))
    out = torch.empty((M, N), device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    moe.mxfp4_matmul_ex(*a, *b, out, d_status=st, test_timeout_cta=cta)
    return int(st), out, value(*a), value(*b)


# (M, N, K, tiles): less than the two meetings of a cluster cost would be saved
@pytest.mark.parametrize("M,N,K,tiles", [(16, 256, 1024, 2), (64, 300, 1536, 3), (100, 130, 2048, 2),
                                         (300, 300, 1024, 9), (128, 2880, 512, 23)])
def test_short_contractions_are_not_shared(cuda_device, M, N, K, tiles):
    st, out, a, b = run(cuda_device, M, N, K, tiles)  # CTAs 0 to tiles - 1 exist
    assert st == moe.MOE_OK
    want = a @ b.T
    assert bool(((out.double() - want).abs() <= product_bound(a.abs() @ b.abs().T, K, 1.0, out.dtype,
                                                             want)).all())


@pytest.mark.parametrize("M,N,K,tiles", [(16, 256, 4096, 2), (64, 300, 8192, 3), (100, 130, 4096, 2),
                                         (4, 2880, 2880, 23)])
def test_long_contractions_are_shared(cuda_device, M, N, K, tiles):
    assert run(cuda_device, M, N, K, tiles)[0] == moe.MOE_ERR_TIMEOUT


@pytest.mark.parametrize("counts,M,N", [([4096, 32, 0, 700, 1, 128, 129, 64], 256, 256),
                                        ([1024] * 8, 256, 256), ([0, 2900, 1500], 40, 200),
                                        ([5, 0, 3500], 100, 130)])
def test_weight_gradients_of_short_and_long_groups(cuda_device, counts, M, N):
    # a cluster shares a long group's positions and leaves a short one's to one CTA
    gen = torch.Generator(device=cuda_device).manual_seed(M + N)
    E, S = len(counts), sum(counts)
    P = moe.mxfp4_transposed_width(S, E)
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32).to(cuda_device)
    a, b = random_mx(gen, (M, P)), random_mx(gen, (N, P))
    outs = []
    for _ in range(3):
        out = torch.full((E, M, N), 77.0, device=cuda_device)
        moe.mxfp4_matmul_grouped_wgrad(*a, *b, off, out)
        outs.append(out)
    av, bv, p = value(*a), value(*b), 0
    for e, c in enumerate(counts):
        n = (c + 127) // 128 * 128
        # no quantiser has zeroed these pads: the sum takes steps of 64 positions
        k = slice(p, p + (c + 63) // 64 * 64)
        want = av[:, k] @ bv[:, k].T
        bound = product_bound(av[:, k].abs() @ bv[:, k].abs().T, max(n, 1), 1.0, out.dtype, want)
        assert bool(((outs[0][e].double() - want).abs() <= bound).all())
        p += n
    assert all(torch.equal(o, outs[0]) for o in outs)
