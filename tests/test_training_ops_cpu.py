"""Host-side refusals of the MXFP4 products, the transposed quantiser and the
gradients of the combine and the sort (nothing reaches a device here)."""
import pytest
import torch

import mxfp4_quantised_mixture_b200 as moe

L = moe.lib
SHAPE, ARG, OK = moe.MOE_ERR_SHAPE, moe.MOE_ERR_INVALID_ARG, moe.MOE_OK


def test_transposed_width():
    w = moe.mxfp4_transposed_width
    assert [w(r) for r in (0, 1, 31, 32, 33, 2880)] == [0, 32, 32, 32, 64, 2880]
    assert w(0, 1) == 0 and w(1, 1) == 128 and w(128, 1) == 128 and w(129, 1) == 256
    assert w(-1) == 0 and w(5, 257) == 0 and w(5, -1) == 0
    # holds every split of the rows into E groups, and the worst split needs all of it
    for rows, E in [(1, 3), (130, 2), (512, 128), (7, 256), (1000, 5)]:
        room = w(rows, E)
        worst = [1] * min(rows, E - 1)
        worst += [rows - sum(worst)]
        assert sum((c + 127) // 128 * 128 for c in worst) <= room


def test_matmul_refusals():
    def call(a=16, sa=16, b=16, sb=16, M=4, N=8, K=64, out=16, kind=0, st=None):
        return L.mxfp4_matmul(a, sa, b, sb, M, N, K, 1.0, out, kind, st, None)

    assert call(K=48) == SHAPE and call(K=0) == SHAPE and call(K=(1 << 24) + 32) == SHAPE
    assert call(M=-1) == SHAPE and call(N=-1) == SHAPE and call(M=(1 << 27) + 1) == SHAPE
    assert call(M=0) == OK and call(N=0) == OK
    assert call(a=None) == ARG and call(sb=None) == ARG and call(out=None) == ARG
    assert call(a=24) == ARG and call(out=8) == ARG and call(st=18) == ARG
    assert call(kind=2) == ARG and call(kind=-1) == ARG


def test_grouped_refusals():
    def call(off=16, E=4, S=8, N=8, K=64, out=16, kind=0):
        return L.mxfp4_matmul_grouped(16, 16, off, E, 16, 16, S, N, K, 1.0, out, kind, None, None)

    assert call(E=0) == SHAPE and call(E=257) == SHAPE and call(S=-1) == SHAPE
    assert call(N=(1 << 26)) == SHAPE and call(K=33) == SHAPE
    assert call(S=0) == OK and call(N=0) == OK
    assert call(off=None) == ARG and call(off=20) == ARG and call(kind=5) == ARG


def test_wgrad_refusals():
    def call(off=16, E=4, M=8, N=8, P=512, out=16, a=16):
        return L.mxfp4_matmul_grouped_wgrad(a, 16, 16, 16, off, E, M, N, P, 1.0, out, 1, None, None)

    assert call(P=96) == SHAPE and call(P=-128) == SHAPE and call(E=0) == SHAPE
    assert call(M=1 << 26) == SHAPE and call(N=-1) == SHAPE
    assert call(M=0) == OK and call(N=0) == OK
    assert call(off=None) == ARG and call(a=None) == ARG and call(out=None, P=0) == ARG


def test_transposed_quantiser_refusals():
    def call(w=16, batch=1, rows=8, cols=16, q=16, s=16, st=None):
        return L.mxfp4_quantize_transposed(w, batch, rows, cols, q, s, st, None)

    assert call(cols=12) == SHAPE and call(cols=0) == SHAPE and call(rows=-1) == SHAPE
    assert call(batch=-1) == SHAPE and call(rows=1 << 30, cols=1 << 20) == SHAPE
    assert call(batch=0) == OK and call(rows=0) == OK
    assert call(w=None) == ARG and call(q=24) == ARG and call(st=18) == ARG

    def grouped(off=16, E=2, rows=8, cols=16, w=16):
        return L.mxfp4_quantize_transposed_grouped(w, rows, cols, off, E, 16, 16, None, None)

    assert grouped(E=0) == SHAPE and grouped(E=257) == SHAPE and grouped(cols=4) == SHAPE
    assert grouped(off=None) == ARG and grouped(off=20) == ARG and grouped(w=None) == ARG
    assert grouped(rows=0, E=1) == OK


def test_gradient_refusals():
    sh = moe.make_shape(4, 8, 2, 128, 128)
    cb, pb = L.moe_combine_backward, L.moe_permute_backward
    bad = moe.make_shape(4, 8, 2, 100, 128)
    assert cb(16, 16, 16, 16, bad, 16, 16, 16, None) == SHAPE
    assert pb(16, 16, bad, 16, None, None, None, None) == SHAPE
    empty = moe.make_shape(0, 8, 2, 128, 128)
    assert cb(None, None, None, None, empty, None, None, None, None) == OK
    assert pb(None, None, empty, None, None, None, None, None) == OK
    assert cb(None, 16, 16, 16, sh, 16, 16, 16, None) == ARG
    assert cb(16, 16, 16, 16, sh, None, 16, 16, None) == ARG
    assert cb(16, None, 16, 16, sh, 16, 16, None, None) == ARG  # dtopk_w needs y_perm
    assert cb(16, None, 16, 16, sh, 16, None, 16, None) == ARG  # so does dscore
    assert cb(16, 16, 20, 16, sh, 16, 16, 16, None) == ARG
    assert pb(16, None, sh, 16, None, None, None, None) == ARG
    # the router's three arguments: all or none
    for args in [(16, None, None), (None, 16, None), (None, None, 16), (16, 16, None), (16, None, 16)]:
        assert pb(16, 16, sh, 16, *args, None) == ARG
    assert pb(16, 16, sh, 24, None, None, None, None) == ARG


def test_binding_refuses_shapes_that_contradict():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    off = torch.zeros(5, dtype=torch.int32)
    out = torch.zeros((4, 8))
    good = (u8(4, 32), u8(4, 2), u8(8, 32), u8(8, 2))
    for i, wrong in [(0, u8(4, 16)), (1, u8(4, 4)), (2, u8(9, 32)), (3, u8(8, 3)),
                     (0, torch.zeros((4, 32), dtype=torch.int32))]:
        args = list(good)
        args[i] = wrong
        with pytest.raises(ValueError, match="belong together"):
            moe.mxfp4_matmul(*args, out)
    with pytest.raises(ValueError, match="CUDA device"):  # host tensors of fitting shapes
        moe.mxfp4_matmul(*good, out)
    with pytest.raises(ValueError):
        moe.mxfp4_matmul(*good, torch.zeros((4, 8), dtype=torch.float16))
    with pytest.raises(ValueError, match="belong together"):  # 4 groups need 4 matrices
        moe.mxfp4_matmul_grouped(*good[:2], off, u8(3, 8, 32), u8(3, 8, 2), out)
    with pytest.raises(ValueError, match="belong together"):
        moe.mxfp4_matmul_grouped_wgrad(u8(4, 64), u8(4, 4), u8(8, 64), u8(8, 4), off,
                                       torch.zeros((3, 4, 8)))
    with pytest.raises(ValueError, match="belong together"):
        moe.mxfp4_quantize_transposed(torch.zeros((40, 16), dtype=torch.bfloat16), u8(16, 16), u8(16, 1))
    with pytest.raises(ValueError, match="belong together"):
        moe.mxfp4_quantize_transposed_grouped(torch.zeros((40, 16), dtype=torch.bfloat16), off,
                                              u8(16, 32), u8(16, 2))


def test_binding_refuses_gradient_shapes_that_contradict():
    sh = moe.make_shape(4, 8, 2, 128, 128)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    pos, w = torch.zeros(8, dtype=torch.int32), torch.zeros((4, 2))
    good = [bf(4, 128), bf(8, 128), pos, w, sh, bf(8, 128), w, w]
    for i, wrong in [(0, bf(5, 128)), (1, bf(4, 128)), (2, pos[:7]), (3, torch.zeros((2, 4))),
                     (5, bf(8, 64)), (6, torch.zeros((4, 3))), (2, pos.long())]:
        args = list(good)
        args[i] = wrong
        with pytest.raises(ValueError, match="belong together"):
            moe.moe_combine_backward(*args)
    with pytest.raises(ValueError, match="CUDA device"):
        moe.moe_combine_backward(*good)
    good = [bf(8, 128), pos, sh, bf(4, 128), torch.zeros((4, 2), dtype=torch.int32), w, bf(8, 128)]
    for i, wrong in [(0, bf(4, 128)), (1, pos.float()), (3, bf(4, 64)), (4, pos), (5, torch.zeros((4, 1))),
                     (6, bf(7, 128))]:
        args = list(good)
        args[i] = wrong
        with pytest.raises(ValueError, match="belong together"):
            moe.moe_permute_backward(*args)
    with pytest.raises(ValueError, match="CUDA device"):
        moe.moe_permute_backward(*good)


def test_well_formed_calls_fail_cleanly_without_a_device():
    if torch.cuda.is_available():
        pytest.skip("its placeholder pointers must never reach a device")
    no_device = (moe.MOE_ERR_CUDA, moe.MOE_ERR_UNSUPPORTED)
    sh = moe.make_shape(4, 8, 2, 128, 128)
    assert L.mxfp4_matmul(16, 16, 16, 16, 4, 8, 64, 1.0, 16, 0, None, None) in no_device
    assert L.mxfp4_matmul_grouped(16, 16, 16, 4, 16, 16, 8, 8, 64, 1.0, 16, 0, None, None) in no_device
    assert L.mxfp4_matmul_grouped_wgrad(16, 16, 16, 16, 16, 4, 8, 8, 512, 1.0, 16, 1, None, None) in no_device
    assert L.mxfp4_quantize_transposed(16, 1, 8, 16, 16, 16, None, None) in no_device
    assert L.mxfp4_quantize_transposed_grouped(16, 8, 16, 16, 2, 16, 16, None, None) in no_device
    assert L.moe_combine_backward(16, 16, 16, 16, sh, 16, 16, 16, None) in no_device
    assert L.moe_permute_backward(16, 16, sh, 16, None, None, None, None) in no_device
