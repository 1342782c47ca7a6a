"""The transposed quantiser, the gradients of the combine and of the sort, and
a forward and backward pass of an expert layer put together from them."""
import numpy as np
import pytest
import torch

import mxfp4_quantised_mixture_b200 as moe
import oracle
from mx_plain import behind_untouched, guarded, product_bound, value

pytestmark = pytest.mark.gpu

HALF16 = 2.0 ** -8   # half a step of bf16, relative
HALF32 = 2.0 ** -24  # half a step of fp32, relative


def u8(shape, dev, fill=0):
    return torch.full(shape, fill, dtype=torch.uint8, device=dev)


def normal(gen, shape, sigma=1.0):
    return (torch.randn(shape, generator=gen, device=gen.device) * sigma).to(torch.bfloat16)


def generator(dev, seed):
    return torch.Generator(device=dev).manual_seed(seed)


def oracle_quantise(w):
    """Bytes of the oracle's quantiser on a CPU copy of w [rows][K]."""
    q, s, bad = oracle.mxfp4_quantize(w.contiguous().cpu().view(torch.int16).numpy().view(np.uint16))
    assert bad == 0
    return torch.from_numpy(q), torch.from_numpy(s)


# ------------------------------------------------------ transposed quantiser

@pytest.mark.parametrize("batch,R,C", [(1, 1, 8), (1, 31, 16), (2, 33, 24), (1, 128, 128), (3, 64, 136),
                                       (1, 129, 264), (2, 320, 8), (1, 1000, 320), (5, 127, 120)])
def test_transposed_equals_quantising_the_transpose(cuda_device, batch, R, C):
    gen = generator(cuda_device, R * C + batch)
    w = normal(gen, (batch, R, C)) * torch.exp2(torch.randint(-20, 20, (batch, R, C), generator=gen,
                                                              device=cuda_device)).to(torch.bfloat16)
    w[:, :, 3] = 0
    P = moe.mxfp4_transposed_width(R)
    assert P == (R + 31) // 32 * 32
    q, qw = guarded((batch, C, P // 2), torch.uint8, cuda_device, 0xAB)
    s, sw = guarded((batch, C, P // 32), torch.uint8, cuda_device, 0xAB)
    st = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    moe.mxfp4_quantize_transposed(w, q, s, st)
    assert int(st) == 0
    t = torch.nn.functional.pad(w.transpose(1, 2), (0, P - R)).reshape(batch * C, P)
    oq, os_ = oracle_quantise(t)
    assert torch.equal(s.cpu().view(-1, P // 32), os_) and torch.equal(q.cpu().view(-1, P // 2), oq)
    assert behind_untouched(q, qw, 0xAB) and behind_untouched(s, sw, 0xAB)


@pytest.mark.parametrize("counts,C", [([1], 8), ([0, 31, 0, 128, 129, 5], 24), ([300], 136), ([0, 0], 16),
                                      ([1] * 256, 40), ([700, 0, 64], 264)])
def test_grouped_transposed(cuda_device, counts, C):
    S, E = sum(counts), len(counts)
    before, behind = 2, 3  # rows in no group: never read (they hold NaN)
    gen = generator(cuda_device, S + C)
    w = torch.full((before + S + behind, C), float("nan"), dtype=torch.bfloat16, device=cuda_device)
    w[before:before + S] = normal(gen, (S, C))
    off = (torch.tensor([0] + counts).cumsum(0) + before).to(torch.int32).to(cuda_device)
    P = moe.mxfp4_transposed_width(S + before + behind, E)
    assert P % 128 == 0 and P >= sum((c + 127) // 128 * 128 for c in counts)
    q, s = u8((C, P // 2), cuda_device, 0xAB), u8((C, P // 32), cuda_device, 0xAB)
    st = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    moe.mxfp4_quantize_transposed_grouped(w, off, q, s, st)
    assert int(st) == 0
    p, r = 0, before
    for c in counts:
        n = (c + 127) // 128 * 128
        if n:
            t = torch.nn.functional.pad(w[r:r + c].T, (0, n - c))
            oq, os_ = oracle_quantise(t)
            assert torch.equal(q[:, p // 2:(p + n) // 2].cpu(), oq)
            assert torch.equal(s[:, p // 32:(p + n) // 32].cpu(), os_)
        p, r = p + n, r + c
    # positions behind the last group stay as they were
    assert bool((q[:, p // 2:] == 0xAB).all()) and bool((s[:, p // 32:] == 0xAB).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_transposed_flags_nonfinite_input(cuda_device, bad):
    w = torch.ones((70, 16), dtype=torch.bfloat16, device=cuda_device)
    w[69, 5] = bad
    P = moe.mxfp4_transposed_width(70)
    st = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    moe.mxfp4_quantize_transposed(w, u8((16, P // 2), cuda_device), u8((16, P // 32), cuda_device), st)
    assert int(st) == moe.MOE_ERR_NONFINITE


def test_transposed_large_against_the_row_quantiser(cuda_device):
    gen = generator(cuda_device, 3)
    w = normal(gen, (3, 2880, 1440), 0.02)
    q, s = u8((3, 1440, 1440), cuda_device), u8((3, 1440, 90), cuda_device)
    moe.mxfp4_quantize_transposed(w, q, s)
    rq, rs = u8((3, 1440, 1440), cuda_device), u8((3, 1440, 90), cuda_device)
    moe.mxfp4_quantize(w.transpose(1, 2).contiguous(), rq, rs)
    assert torch.equal(q, rq) and torch.equal(s, rs)


# ------------------------------------------------ gradients of combine and sort

def positions(gen, T, k, dropped=0.0):
    """slot_pos of a random routing; dropped slots get -1 (or a position past the end)."""
    S = T * k
    pos = torch.randperm(S, generator=gen, device=gen.device).to(torch.int32)
    if dropped:
        drop = torch.rand(S, generator=gen, device=gen.device) < dropped
        pos = torch.where(drop, torch.where(pos % 2 == 0, -1, S + 5).to(torch.int32), pos)
    return pos


SHAPES = [(1, 8, 1, 128), (3, 8, 8, 192), (17, 5, 4, 2880), (100, 32, 4, 320), (64, 7, 3, 1024),
          (2500, 16, 2, 128), (5, 256, 7, 16384), (9, 6, 5, 640), (11, 9, 6, 256)]


@pytest.mark.parametrize("dropped", [0.0, 0.3])
@pytest.mark.parametrize("T,E,k,D", SHAPES)
def test_combine_backward(cuda_device, T, E, k, D, dropped):
    gen = generator(cuda_device, T * D + k)
    S = T * k
    dout, y = normal(gen, (T, D), 0.1), normal(gen, (S, D))
    pos = positions(gen, T, k, dropped)
    w = torch.softmax(torch.randn((T, k), generator=gen, device=cuda_device), 1)
    dy, whole = guarded((S, D), torch.bfloat16, cuda_device, 3.0)
    dw = torch.full((T, k), 9.0, device=cuda_device)
    ds = torch.full((T, k), 9.0, device=cuda_device)
    sh = moe.make_shape(T, E, k, D, D)
    moe.moe_combine_backward(dout, y, pos, w, sh, dy, dw, ds)
    p = pos.view(T, k).long()
    live = (p >= 0) & (p < S)
    terms = dout.double()[:, None] * y.double()[p.clamp(0, S - 1)] * live[..., None]
    want_dw = terms.sum(-1)
    # D fp32 fused additions, each off by half a step of a sum below the magnitudes'
    err_dw = D * HALF32 * terms.abs().sum(-1) + 1e-37
    assert bool(((dw.double() - want_dw).abs() <= err_dw).all())
    wd = w.double()
    want_ds = wd * (want_dw - (wd * want_dw).sum(1, keepdim=True))
    size = wd * (want_dw.abs() + (wd * want_dw.abs()).sum(1, keepdim=True))
    err_ds = wd * (err_dw + (wd * err_dw).sum(1, keepdim=True)) + (k + 3) * HALF32 * size + 1e-37
    assert bool(((ds.double() - want_ds).abs() <= err_ds).all())
    want_dy = torch.full((S, D), 3.0, dtype=torch.float64, device=cuda_device)
    want_dy[p[live]] = (wd[..., None] * dout.double()[:, None])[live]
    # one fp32 rounding, then one bf16 rounding
    assert bool(((dy.double() - want_dy).abs() <= (HALF16 + 2 * HALF32) * want_dy.abs() + 1e-37).all())
    assert behind_untouched(dy, whole, 3.0)


def test_combine_backward_optional_outputs(cuda_device):
    gen = generator(cuda_device, 4)
    T, k, D = 33, 4, 256
    sh = moe.make_shape(T, 8, k, D, D)
    dout, y, pos = normal(gen, (T, D)), normal(gen, (T * k, D)), positions(gen, T, k)
    w = torch.softmax(torch.randn((T, k), generator=gen, device=cuda_device), 1)
    full = [torch.empty((T * k, D), dtype=torch.bfloat16, device=cuda_device),
            torch.empty((T, k), device=cuda_device), torch.empty((T, k), device=cuda_device)]
    moe.moe_combine_backward(dout, y, pos, w, sh, *full)
    dy, a, b = torch.empty_like(full[0]), torch.empty_like(full[1]), torch.empty_like(full[1])
    moe.moe_combine_backward(dout, None, pos, w, sh, dy)
    assert torch.equal(dy, full[0])
    moe.moe_combine_backward(dout, y, pos, w, sh, dy, a)
    moe.moe_combine_backward(dout, y, pos, w, sh, dy, None, b)
    assert torch.equal(a, full[1]) and torch.equal(b, full[2])


@pytest.mark.parametrize("router", [False, True])
@pytest.mark.parametrize("dropped", [0.0, 0.3])
@pytest.mark.parametrize("T,E,k,D", SHAPES)
def test_permute_backward(cuda_device, T, E, k, D, dropped, router):
    gen = generator(cuda_device, T * D + k + 1)
    S = T * k
    dxp = normal(gen, (S, D), 0.1)
    pos = positions(gen, T, k, dropped)
    idx = torch.rand((T, E), generator=gen, device=cuda_device).argsort(1)[:, :k].to(torch.int32).contiguous()
    if dropped:
        idx[0, 0] = E + 3  # outside: contributes nothing
    ds = torch.randn((T, k), generator=gen, device=cuda_device) * 0.1
    wr = normal(gen, (E, D), D ** -0.5)
    dx, whole = guarded((T, D), torch.bfloat16, cuda_device, 3.0)
    moe.moe_permute_backward(dxp, pos, moe.make_shape(T, E, k, D, D), dx,
                             *((idx, ds, wr) if router else ()))
    p = pos.view(T, k).long()
    live = (p >= 0) & (p < S)
    terms = dxp.double()[p.clamp(0, S - 1)] * live[..., None]
    if router:
        inside = (idx < E)[..., None]
        terms = torch.cat([terms, ds.double()[..., None] * wr.double()[idx.long().clamp(max=E - 1)] * inside], 1)
    want = terms.sum(1)
    acc = 2 * k * HALF32 * terms.abs().sum(1)
    assert bool(((dx.double() - want).abs() <= acc + HALF16 * (want.abs() + acc) + 1e-37).all())
    assert behind_untouched(dx, whole, 3.0)


def test_gradients_against_differences(cuda_device):
    # L(scores, y, x) = <combine(softmax(scores), y), g> and the sort's gather: central differences
    # of the 64-bit forms in random directions
    gen = generator(cuda_device, 6)
    T, k, D, E = 12, 4, 128, 8
    S = T * k
    g, y, pos = normal(gen, (T, D)), normal(gen, (S, D)), positions(gen, T, k)
    sc = torch.randn((T, k), generator=gen, device=cuda_device)
    w = torch.softmax(sc, 1)
    sh = moe.make_shape(T, E, k, D, D)
    dy = torch.empty((S, D), dtype=torch.bfloat16, device=cuda_device)
    dw, ds = torch.empty((T, k), device=cuda_device), torch.empty((T, k), device=cuda_device)
    moe.moe_combine_backward(g, y, pos, w, sh, dy, dw, ds)
    p = pos.view(T, k).long()

    def loss(weights, rows):
        return ((weights[..., None] * rows[p]).sum(1) * g.double()).sum()

    def soft(s):
        return torch.softmax(s, 1)

    h = 2.0 ** -12
    vs = torch.randn((T, k), generator=gen, device=cuda_device, dtype=torch.float64)
    vy = torch.randn((S, D), generator=gen, device=cuda_device, dtype=torch.float64)
    s64, y64 = sc.double(), y.double()
    diff = (loss(soft(s64 + h * vs), y64) - loss(soft(s64 - h * vs), y64)) / (2 * h)
    # the softmax's third derivative is below 1 and h^2 / 6 below 2^-26; fp32 weights and sums: below
    # 2^-14 of the magnitudes at these sizes
    scale = (vs.abs() * (w.double()[..., None] * y64[p] * g.double()[:, None]).abs().sum(-1)).sum()
    assert abs(float((ds.double() * vs).sum() - diff)) <= 2.0 ** -14 * float(scale)
    diff = (loss(w.double(), y64 + h * vy) - loss(w.double(), y64 - h * vy)) / (2 * h)
    size = float((dy.double() * vy).abs().sum())
    assert abs(float((dy.double() * vy).sum() - diff)) <= 2 * HALF16 * size
    # the gather: <x[t(p)], dxp> is linear in x
    dx = torch.empty((T, D), dtype=torch.bfloat16, device=cuda_device)
    moe.moe_permute_backward(dy, pos, sh, dx)
    vx = torch.randn((T, D), generator=gen, device=cuda_device, dtype=torch.float64)
    rows = vx[:, None].expand(T, k, D)
    want = float((rows * dy.double()[p]).sum())
    size = float((rows * dy.double()[p]).abs().sum())
    assert abs(float((dx.double() * vx).sum()) - want) <= 2 * HALF16 * size


def test_training_ops_in_a_graph_on_another_stream(cuda_device):
    gen = generator(cuda_device, 7)
    T, k, D, E = 50, 3, 320, 6
    S = T * k
    sh = moe.make_shape(T, E, k, D, D)
    dout, y, pos = normal(gen, (T, D)), normal(gen, (S, D)), positions(gen, T, k)
    w = torch.softmax(torch.randn((T, k), generator=gen, device=cuda_device), 1)

    def run():
        dy = torch.empty((S, D), dtype=torch.bfloat16, device=cuda_device)
        dw = torch.empty((T, k), device=cuda_device)
        dx = torch.empty((T, D), dtype=torch.bfloat16, device=cuda_device)
        moe.moe_combine_backward(dout, y, pos, w, sh, dy, dw)
        moe.moe_permute_backward(dy, pos, sh, dx)
        return dy, dw, dx

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run()
    dout.copy_(normal(gen, (T, D)))
    g.replay()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        want = run()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


# ----------------------------------------------------- a whole step, put together

@pytest.mark.parametrize("T,E,k,D,F", [(40, 8, 2, 128, 192), (300, 4, 4, 256, 128), (7, 16, 1, 192, 320)])
def test_forward_and_backward_of_an_expert_layer(cuda_device, T, E, k, D, F):
    """Route, sort, quantise, gate/up product, SwiGLU, quantise, down product, combine; then every
    gradient back to x, the scores and both weights.  Each call is compared with the 64-bit form of
    its step on the same inputs (a quantisation in between rounds differences up to whole steps)."""
    gen = generator(cuda_device, T + D)
    S, dev = T * k, cuda_device
    x, wr = normal(gen, (T, D)), normal(gen, (E, D), D ** -0.5)
    wgu, wdn = normal(gen, (E, 2 * F, D), 0.1), normal(gen, (E, D, F), 0.1)
    g = normal(gen, (T, D), 0.1)
    sh = moe.make_shape(T, E, k, D, F)

    def mx(t):
        q, s = u8(t.shape[:-1] + (t.shape[-1] // 2,), dev), u8(t.shape[:-1] + (t.shape[-1] // 32,), dev)
        moe.mxfp4_quantize(t.contiguous(), q, s)
        return q, s

    def mx_t(t):
        P = moe.mxfp4_transposed_width(t.shape[-2])
        shape = t.shape[:-2] + (t.shape[-1],)
        q, s = u8(shape + (P // 2,), dev), u8(shape + (P // 32,), dev)
        moe.mxfp4_quantize_transposed(t, q, s)
        return q, s

    def mx_g(t):
        P = moe.mxfp4_transposed_width(S, E)
        q, s = u8((t.shape[1], P // 2), dev), u8((t.shape[1], P // 32), dev)
        moe.mxfp4_quantize_transposed_grouped(t, off, q, s)
        return q, s

    def grouped(a, b, n):
        out = torch.empty((S, n), dtype=torch.bfloat16, device=dev)
        moe.mxfp4_matmul_grouped(*a, off, *b, out)
        av, bv = value(*a), value(*b)
        for e in range(E):
            rows = slice(bounds[e], bounds[e + 1])
            want = av[rows] @ bv[e].T
            bound = product_bound(av[rows].abs() @ bv[e].abs().T, av.shape[1], 1.0, out.dtype, want)
            assert bool(((out[rows].double() - want).abs() <= bound).all())
        return out

    def wgrad(a, b):
        out = torch.empty((E, a[0].shape[0], b[0].shape[0]), device=dev)
        moe.mxfp4_matmul_grouped_wgrad(*a, *b, off, out)
        av, bv, p = value(*a), value(*b), 0
        for e in range(E):
            n = (bounds[e + 1] - bounds[e] + 127) // 128 * 128
            want = av[:, p:p + n] @ bv[:, p:p + n].T
            bound = product_bound(av[:, p:p + n].abs() @ bv[:, p:p + n].abs().T, n, 1.0, out.dtype, want)
            assert bool(((out[e].double() - want).abs() <= bound).all())
            p += n
        return out

    idx = torch.empty((T, k), dtype=torch.int32, device=dev)
    w = torch.empty((T, k), device=dev)
    moe.moe_router_topk(x, wr, k, idx, w)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    off = torch.empty(E + 1, dtype=torch.int32, device=dev)
    order, pos = (torch.empty(S, dtype=torch.int32, device=dev) for _ in range(2))
    xp = torch.empty((S, D), dtype=torch.bfloat16, device=dev)
    moe.moe_permute(idx, x, sh, counts, off, order, pos, xp)
    bounds = off.tolist()
    gu = grouped(mx(xp), mx(wgu), 2 * F)
    gate, up = gu.float()[:, :F], gu.float()[:, F:]
    h = (torch.nn.functional.silu(gate) * up).to(torch.bfloat16)
    y = grouped(mx(h), mx(wdn), D)
    out = torch.empty((T, D), dtype=torch.bfloat16, device=dev)
    moe.moe_combine(y, pos, w, sh, out)

    dy = torch.empty((S, D), dtype=torch.bfloat16, device=dev)
    ds = torch.empty((T, k), device=dev)
    moe.moe_combine_backward(g, y, pos, w, sh, dy, None, ds)
    dh = grouped(mx(dy), mx_t(wdn), F).float()
    d_wdn = wgrad(mx_g(dy), mx_g(h))
    sig = torch.sigmoid(gate)
    dgate = dh * up * sig * (1 + gate * (1 - sig))
    dgu = torch.cat([dgate, dh * gate * sig], 1).to(torch.bfloat16)
    dxp = grouped(mx(dgu), mx_t(wgu), D)
    d_wgu = wgrad(mx_g(dgu), mx_g(xp))
    dx = torch.empty((T, D), dtype=torch.bfloat16, device=dev)
    moe.moe_permute_backward(dxp, pos, sh, dx, idx, ds, wr)
    assert d_wdn.shape == wdn.shape and d_wgu.shape == wgu.shape

    # the whole step against autograd through the unquantised layer: MXFP4 rounds every element to
    # within a quarter of itself, so the directions agree though the values differ
    leaves = [t.double().requires_grad_() for t in (x, wgu, wdn)]
    x64, gu64, dn64 = leaves
    p = pos.view(T, k).long()
    sc = (x64 @ wr.double().T).gather(1, idx.long())
    tok = order.long() // k
    rows = x64[tok]
    parts = []
    for e in range(E):
        r = rows[bounds[e]:bounds[e + 1]]
        a = r @ gu64[e].T
        parts.append((torch.nn.functional.silu(a[:, :F]) * a[:, F:]) @ dn64[e].T)
    full = (torch.softmax(sc, 1)[..., None] * torch.cat(parts)[p]).sum(1)
    (full * g.double()).sum().backward()
    for got, want in ((out, full.detach()), (dx, x64.grad), (d_wgu, gu64.grad), (d_wdn, dn64.grad)):
        cos = (got.double() * want).sum() / (got.double().norm() * want.norm())
        assert float(cos) > 0.9
