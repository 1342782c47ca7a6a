"""The bounded-wait failure path of the MXFP4 product kernels, without a GPU fault.

mxfp4_matmul_ex(test_timeout_cta=c) makes the MMA warp of CTA c wait, with a
short limit, on a barrier that nothing completes, so it gives up as a real
timeout would: the CTA records MOE_ERR_TIMEOUT in the device status word, its
roles leave their loops, it waits for its own copies and MMAs, meets its cluster,
frees its tensor memory and exits.  The context stays usable: the next call's
result is the earlier one bit for bit."""
import pytest
import torch

import mxfp4_quantised_mixture_b200 as moe
from mx_plain import behind_untouched, guarded, random_mx

pytestmark = pytest.mark.gpu

FILL = 77.0

# (M, N, K, CTA that gives up)
ONE_CTA = [(16, 20000, 512, 0), (64, 25600, 1056, 3), (128, 19200, 2080, 147)]
CLUSTER = [(16, 256, 4096, 0), (16, 256, 4096, 3), (60, 300, 8192, 7), (100, 130, 16384, 2)]
PAIR = [(1500, 1301, 1120, 0), (1500, 1301, 1120, 1), (4000, 2600, 4128, 2), (4000, 2600, 4128, 147),
        (1300, 1300, 32, 5)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K,cta", ONE_CTA + CLUSTER + PAIR)
def test_timeout_is_reported_and_the_next_call_is_exact(cuda_device, M, N, K, cta, dtype):
    gen = torch.Generator(device=cuda_device).manual_seed(M + N + K)
    a, b = random_mx(gen, (M, K)), random_mx(gen, (N, K))

    def call(fail):
        out, whole = guarded((M, N), dtype, cuda_device, FILL)
        st = torch.zeros(1, dtype=torch.int32, device=cuda_device)
        moe.mxfp4_matmul_ex(*a, *b, out, d_status=st, test_timeout_cta=fail)
        torch.cuda.synchronize()
        assert behind_untouched(out, whole, FILL)
        return int(st), out

    st, first = call(-1)
    assert st == moe.MOE_OK
    st, _ = call(cta)
    assert st == moe.MOE_ERR_TIMEOUT
    for _ in range(2):
        st, again = call(-1)
        assert st == moe.MOE_OK and torch.equal(first, again)
