"""Products of two MXFP4 matrices (mxfp4_matmul, mxfp4_matmul_grouped,
mxfp4_matmul_grouped_wgrad) against 64-bit products of the values the codes
stand for ("MXFP4-based MoE technical review", section 2)."""
import pytest
import torch

import mxfp4_quantised_mixture_b200 as moe
from mx_plain import behind_untouched, guarded, product_bound, random_mx, value

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float32]
FILL = 77.0


def generator(dev, seed):
    return torch.Generator(device=dev).manual_seed(seed)


def status(dev):
    return torch.zeros(1, dtype=torch.int32, device=dev)


def assert_product(out, a, b, K, alpha):
    """out against alpha a b^T, a and b float64."""
    want = alpha * (a @ b.transpose(-1, -2))
    bound = product_bound(a.abs() @ b.abs().transpose(-1, -2), K, alpha, out.dtype, want)
    off = (out.double() - want).abs()
    assert bool((off <= bound).all()), (float((off / bound).max()), out.shape)


def offsets_of(counts, dev, start=0):
    t = torch.tensor([start] + list(counts)).cumsum(0)
    return t.to(torch.int32).to(dev)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 128, 64), (3, 130, 96), (16, 17, 288),
                                   (17, 2880, 2880), (33, 100, 1056), (64, 128, 1024),
                                   (65, 257, 1120), (128, 128, 256), (129, 384, 4128),
                                   (200, 96, 64), (225, 129, 2080), (500, 1000, 512),
                                   (1000, 72, 8192), (3, 64, 16416), (700, 5760, 2880)])
def test_dense(cuda_device, M, N, K, dtype):
    gen = generator(cuda_device, M * 31 + N * 7 + K)
    a, b = random_mx(gen, (M, K)), random_mx(gen, (N, K))
    out, whole = guarded((M, N), dtype, cuda_device, FILL)
    st = status(cuda_device)
    moe.mxfp4_matmul(*a, *b, out, d_status=st)
    assert int(st) == 0
    assert_product(out, value(*a), value(*b), K, 1.0)
    assert behind_untouched(out, whole, FILL)


def test_dense_sums_of_equal_scales_are_exact(cuda_device):
    # codes are multiples of 1/2 up to 6: with one scale for all, a sum of K = 2880 products is a
    # multiple of 1/4 below 2880 * 36 < 2^17, so fp32 holds every partial sum exactly
    gen = generator(cuda_device, 5)
    M, N, K = 150, 200, 2880
    a, b = random_mx(gen, (M, K), 0), random_mx(gen, (N, K), 0)
    out = torch.empty((M, N), device=cuda_device)
    moe.mxfp4_matmul(*a, *b, out, alpha=1 / 32)
    assert torch.equal(out.double(), value(*a) @ value(*b).T / 32)


@pytest.mark.parametrize("alpha", [0.0, -2.5, 1 / 32])
def test_alpha(cuda_device, alpha):
    gen = generator(cuda_device, 6)
    a, b = random_mx(gen, (40, 160)), random_mx(gen, (50, 160))
    out = torch.empty((40, 50), device=cuda_device)
    moe.mxfp4_matmul(*a, *b, out, alpha=alpha)
    assert_product(out, value(*a), value(*b), 160, alpha)


def test_every_code_and_block_position(cuda_device):
    # one nonzero element per row of A meets B's element in the same place, and nothing else
    K = 320
    a_q = torch.zeros((K, K // 2), dtype=torch.uint8, device=cuda_device)
    rows = torch.arange(K, device=cuda_device)
    code = (rows % 16).to(torch.uint8)
    a_q[rows, rows // 2] = torch.where(rows % 2 == 0, code, code << 4)
    a_s = (110 + rows[:, None] % 20 + torch.arange(K // 32, device=cuda_device)).to(torch.uint8)
    b = random_mx(generator(cuda_device, 7), (130, K))
    out = torch.empty((K, 130), device=cuda_device)
    moe.mxfp4_matmul(a_q, a_s, *b, out)
    assert torch.equal(out.double(), value(a_q, a_s) @ value(*b).T)


def test_scale_extremes(cuda_device):
    # the smallest and largest scale bytes: 2^-127 * 2^127 is 1; a scale byte 255 is NaN and stays
    # in its own row and column
    K = 64
    a_q = torch.full((4, K // 2), 0x22, dtype=torch.uint8, device=cuda_device)  # all 1.0
    b_q = torch.full((5, K // 2), 0x22, dtype=torch.uint8, device=cuda_device)
    a_s = torch.tensor([0, 127, 254, 255], dtype=torch.uint8, device=cuda_device)[:, None].repeat(1, 2)
    b_s = torch.tensor([254, 127, 0, 120, 130], dtype=torch.uint8, device=cuda_device)[:, None].repeat(1, 2)
    out = torch.empty((4, 5), device=cuda_device)
    moe.mxfp4_matmul(a_q, a_s.contiguous(), b_q, b_s.contiguous(), out)
    assert torch.isnan(out[3]).all()
    assert torch.equal(out[:3].diagonal(), torch.full((3,), 64.0, device=cuda_device))
    assert torch.equal(out[1, 3:], torch.tensor([0.5, 512.0], device=cuda_device))
    # 64 * 2^127 = 2^133 is past fp32's range, 64 * 2^-254 below it
    assert torch.isinf(out[1, 0]) and torch.isinf(out[2, 0]) and float(out[0, 2]) == 0
    assert out[0, [1, 3, 4]].tolist() == [2.0 ** -121, 2.0 ** -128, 2.0 ** -118]


GROUPS = [([0, 5, 0, 1, 130, 0], 100, 96), ([1], 128, 32), ([300, 17], 257, 1056),
          ([8] * 32, 384, 2880), ([0] * 7 + [40], 64, 512), ([3, 0] * 128, 72, 64),
          ([224, 225, 448, 16], 130, 288), ([1000, 1], 200, 2080)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("counts,N,K", GROUPS)
def test_grouped(cuda_device, counts, N, K, dtype):
    E, S = len(counts), sum(counts)
    gen = generator(cuda_device, S + N + K)
    a, b = random_mx(gen, (S, K)), random_mx(gen, (E, N, K))
    out, whole = guarded((S, N), dtype, cuda_device, FILL)
    st = status(cuda_device)
    moe.mxfp4_matmul_grouped(*a, offsets_of(counts, cuda_device), *b, out, d_status=st)
    assert int(st) == 0
    av, lo = value(*a), 0
    for e, c in enumerate(counts):
        if c:
            assert_product(out[lo:lo + c], av[lo:lo + c], value(b[0][e], b[1][e]), K, 1.0)
        lo += c
    assert behind_untouched(out, whole, FILL)


def test_grouped_rows_of_no_group_stay(cuda_device):
    counts, before, behind, N, K = [20, 0, 150], 3, 40, 96, 160
    S = before + sum(counts) + behind
    gen = generator(cuda_device, 8)
    a, b = random_mx(gen, (S, K)), random_mx(gen, (3, N, K))
    out = torch.full((S, N), FILL, device=cuda_device)
    off = offsets_of(counts, cuda_device, before)
    moe.mxfp4_matmul_grouped(*a, off, *b, out)
    assert bool((out[:before] == FILL).all()) and bool((out[-behind:] == FILL).all())
    av = value(*a)
    assert_product(out[3:23], av[3:23], value(b[0][0], b[1][0]), K, 1.0)
    assert_product(out[23:173], av[23:173], value(b[0][2], b[1][2]), K, 1.0)


def test_grouped_without_rows(cuda_device):
    gen = generator(cuda_device, 9)
    a, b = random_mx(gen, (50, 64)), random_mx(gen, (4, 80, 64))
    out = torch.full((50, 80), FILL, device=cuda_device)
    moe.mxfp4_matmul_grouped(*a, torch.zeros(5, dtype=torch.int32, device=cuda_device), *b, out)
    assert bool((out == FILL).all())


WGRAD = [([1], 8, 8), ([0, 5, 0, 33], 72, 40), ([128, 1, 0, 129], 136, 264),
         ([64, 65, 700], 232, 128), ([0] * 3, 16, 24), ([2] * 200, 24, 136), ([2100], 304, 520)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("counts,M,N", WGRAD)
def test_wgrad(cuda_device, counts, M, N, dtype):
    E, S = len(counts), sum(counts)
    P = moe.mxfp4_transposed_width(S, E)
    gen = generator(cuda_device, S + M + N)
    off = offsets_of(counts, cuda_device)
    pair = []
    for C in (M, N):
        # positions that no group owns hold NaN scales: nothing may read them
        q = torch.full((C, P // 2), 0x77, dtype=torch.uint8, device=cuda_device)
        s = torch.full((C, P // 32), 255, dtype=torch.uint8, device=cuda_device)
        w = torch.randn((S, C), generator=gen, device=cuda_device).to(torch.bfloat16)
        moe.mxfp4_quantize_transposed_grouped(w, off, q, s)
        pair += [q, s]
    out, whole = guarded((E, M, N), dtype, cuda_device, FILL)
    st = status(cuda_device)
    moe.mxfp4_matmul_grouped_wgrad(*pair, off, out, alpha=0.5, d_status=st)
    assert int(st) == 0
    p = 0
    for e, c in enumerate(counts):
        n = (c + 127) // 128 * 128
        a = value(pair[0][:, p // 2:(p + n) // 2], pair[1][:, p // 32:(p + n) // 32])
        b = value(pair[2][:, p // 2:(p + n) // 2], pair[3][:, p // 32:(p + n) // 32])
        if c:
            assert_product(out[e], a, b, n, 0.5)
        else:
            assert bool((out[e] == 0).all())
        p += n
    assert behind_untouched(out, whole, FILL)


def test_wgrad_without_any_position(cuda_device):
    empty = [torch.empty((8, 0), dtype=torch.uint8, device=cuda_device) for _ in range(4)]
    out = torch.full((1, 8, 8), FILL, device=cuda_device)
    moe.mxfp4_matmul_grouped_wgrad(*empty, torch.zeros(2, dtype=torch.int32, device=cuda_device), out)
    assert bool((out == 0).all())


def test_transformed_operands(cuda_device):
    # the same random Hadamard transform on both operands: alpha = 1/32 undoes it, and the product
    # is that of the quantised transformed values
    gen = generator(cuda_device, 10)
    M, N, K = 70, 90, 256
    signs = torch.randint(-2 ** 31, 2 ** 31, (K // 32,), generator=gen, device=cuda_device).to(torch.int32)
    sides = []
    for rows in (M, N):
        w = torch.randn((rows, K), generator=gen, device=cuda_device).to(torch.bfloat16)
        q = torch.empty((rows, K // 2), dtype=torch.uint8, device=cuda_device)
        s = torch.empty((rows, K // 32), dtype=torch.uint8, device=cuda_device)
        moe.mxfp4_quantize_sr_rht(w, moe.MOE_QUANT_RHT, signs, 0, q, s)
        sides += [(q, s, w)]
    out = torch.empty((M, N), device=cuda_device)
    moe.mxfp4_matmul(*sides[0][:2], *sides[1][:2], out, alpha=1 / 32)
    a, b = value(*sides[0][:2]), value(*sides[1][:2])
    assert_product(out, a, b, K, 1 / 32)
    plain = sides[0][2].double() @ sides[1][2].double().T
    # E2M1 keeps each element to a quarter of itself or 1/4 of the scale: two operands of K = 256
    # independent errors stay far inside one third of the product's norm
    assert float((out.double() - plain).norm() / plain.norm()) < 1 / 3


def test_repeated_calls_agree_bit_for_bit(cuda_device):
    gen = generator(cuda_device, 11)
    counts = [37, 0, 512, 3, 260, 900]
    a, b = random_mx(gen, (sum(counts), 1120)), random_mx(gen, (6, 700, 1120))
    off = offsets_of(counts, cuda_device)
    first = None
    for _ in range(20):
        out = torch.empty((sum(counts), 700), device=cuda_device)
        moe.mxfp4_matmul_grouped(*a, off, *b, out)
        first = out if first is None else first
        assert torch.equal(out, first)


def test_streams_and_graphs(cuda_device):
    # two captured graphs of products replayed together on two streams, on changed inputs
    gen = generator(cuda_device, 12)
    sides = []
    for n in (300, 900):
        a, b = random_mx(gen, (n, 512)), random_mx(gen, (200, 512))
        sides.append((a, b, torch.empty((n, 200), device=cuda_device)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for (a, b, out), s in zip(sides, streams):
        moe.mxfp4_matmul(*a, *b, out, stream=s)
    torch.cuda.synchronize()
    graphs = []
    for a, b, out in sides:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.mxfp4_matmul(*a, *b, out)
        graphs.append(g)
    for a, b, _ in sides:
        a[0].copy_(random_mx(gen, (a[0].shape[0], 512))[0])
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, b, out in sides:
        assert_product(out, value(*a), value(*b), 512, 1.0)


def test_outputs_past_32_bits(cuda_device):
    # 2^30 < 40000 * 30016 elements, past 2^32 bytes: rows from the start, the middle and the end
    gen = generator(cuda_device, 13)
    M, N, K = 40000, 30016, 64
    a, b = random_mx(gen, (M, K)), random_mx(gen, (N, K))
    out = torch.empty((M, N), device=cuda_device)
    moe.mxfp4_matmul(*a, *b, out)
    for lo in (0, 17777, M - 33):
        rows = slice(lo, lo + 33)
        assert_product(out[rows], value(a[0][rows], a[1][rows]), value(*b), K, 1.0)


@pytest.mark.parametrize("M,N,K", [(1, 2880, 2880), (16, 256, 4096), (100, 130, 16384), (33, 300, 1088)])
def test_few_tiles_share_the_contraction(cuda_device, M, N, K):
    # a cluster of CTAs splits k; the outcome is the same on every call, and the empty sum of a
    # group without positions is zero there too
    gen = generator(cuda_device, M + K)
    a, b = random_mx(gen, (M, K)), random_mx(gen, (N, K))
    outs = []
    for _ in range(5):
        out, whole = guarded((M, N), torch.float32, cuda_device, FILL)
        moe.mxfp4_matmul(*a, *b, out, alpha=2.0)
        assert behind_untouched(out, whole, FILL)
        outs.append(out)
    assert_product(outs[0], value(*a), value(*b), K, 2.0)
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_wgrad_with_few_tiles(cuda_device):
    counts, M, N = [0, 3000, 70], 24, 130
    S, E = sum(counts), len(counts)
    gen = generator(cuda_device, 14)
    off = offsets_of(counts, cuda_device)
    P = moe.mxfp4_transposed_width(S, E)
    pair = []
    for C in (M, N + 6):
        q = torch.empty((C, P // 2), dtype=torch.uint8, device=cuda_device)
        s = torch.empty((C, P // 32), dtype=torch.uint8, device=cuda_device)
        w = torch.randn((S, C), generator=gen, device=cuda_device).to(torch.bfloat16)
        moe.mxfp4_quantize_transposed_grouped(w, off, q, s)
        pair.append((q[:C - 6 * (C != M)].contiguous(), s[:C - 6 * (C != M)].contiguous()))
    out = torch.full((E, M, N), FILL, device=cuda_device)
    moe.mxfp4_matmul_grouped_wgrad(*pair[0], *pair[1], off, out)
    p = 0
    for e, c in enumerate(counts):
        n = (c + 127) // 128 * 128
        a, b = (value(q[:, p // 2:(p + n) // 2], s[:, p // 32:(p + n) // 32]) for q, s in pair)
        assert_product(out[e], a, b, max(n, 1), 1.0)
        p += n


# More than 49 tiles of 128 x 128 run on CTA pairs: widths that fill no tile, odd output widths, k
# that ends inside every kind of step, one and several scale chunks
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [(1500, 1301, 1120), (2000, 1000, 288), (1300, 1300, 32),
                                   (1100, 1111, 4128), (193, 4100, 544), (6500, 130, 96),
                                   (1345, 1537, 2080), (900, 1024, 1024)])
def test_dense_on_pairs(cuda_device, M, N, K, dtype):
    gen = generator(cuda_device, M + N + K)
    a, b = random_mx(gen, (M, K)), random_mx(gen, (N, K))
    out, whole = guarded((M, N), dtype, cuda_device, FILL)
    st = status(cuda_device)
    moe.mxfp4_matmul(*a, *b, out, alpha=0.25, d_status=st)
    assert int(st) == 0
    assert_product(out, value(*a), value(*b), K, 0.25)
    assert behind_untouched(out, whole, FILL)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("counts,N,K", [([300, 17, 0, 700, 193, 1], 2050, 1056),
                                        ([0, 1500, 0], 1301, 160), ([193] * 9, 900, 2880),
                                        ([5, 3000, 0, 1, 64], 1024, 512)])
def test_grouped_on_pairs(cuda_device, counts, N, K, dtype):
    E, S, before, behind = len(counts), sum(counts), 5, 7
    gen = generator(cuda_device, S + N + K)
    a, b = random_mx(gen, (before + S + behind, K)), random_mx(gen, (E, N, K))
    # rows of no group hold NaN scales: no group's rows may meet them
    a[1][:before] = 255
    a[1][-behind:] = 255
    out, whole = guarded((before + S + behind, N), dtype, cuda_device, FILL)
    moe.mxfp4_matmul_grouped(*a, offsets_of(counts, cuda_device, before), *b, out)
    av, lo = value(*a), before
    for e, c in enumerate(counts):
        if c:
            assert_product(out[lo:lo + c], av[lo:lo + c], value(b[0][e], b[1][e]), K, 1.0)
        lo += c
    assert bool((out[:before] == FILL).all()) and bool((out[-behind:] == FILL).all())
    assert behind_untouched(out, whole, FILL)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("counts,M,N", [([130, 0, 700, 64], 1000, 1304), ([1, 0], 1200, 800),
                                        ([2500], 904, 1000), ([64, 65, 63, 0, 1025], 320, 904)])
def test_wgrad_on_pairs(cuda_device, counts, M, N, dtype):
    test_wgrad(cuda_device, counts, M, N, dtype)


def test_pairs_repeat_bit_for_bit_and_share_the_device(cuda_device):
    gen = generator(cuda_device, 15)
    counts = [37, 0, 512, 3, 260, 900]
    a, b = random_mx(gen, (sum(counts), 1120)), random_mx(gen, (6, 1700, 1120))
    off = offsets_of(counts, cuda_device)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [torch.empty((sum(counts), 1700), device=cuda_device) for _ in range(24)]
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        moe.mxfp4_matmul_grouped(*a, off, *b, out, stream=streams[i % 2])
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[0]) for o in outs)
