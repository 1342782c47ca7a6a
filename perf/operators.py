"""Timed cases of the MXFP4 products, their gradients, and the gradients of
the sort by expert and of the weighted way back.

``run`` makes one pass: with ``own`` false in plain torch operations, with
``own`` true through the library.  MXFP4 here is E2M1 codes (two to a byte,
even element in the low nibble) with one E8M0 scale per 32 elements.
"""
import math

import torch

own = False

DEV = "cuda"
OUT = {"bf16": torch.bfloat16, "fp32": torch.float32}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one projection of a few tokens: launch and latency, the weights read once
        {"name": "matmul_few_rows", "op": "matmul", "M": 4, "N": 2880, "K": 2880, "out": "bf16"},
        # a dense projection of a prefill batch, tensor-core bound
        {"name": "matmul_prefill", "op": "matmul", "M": 8192, "N": 5760, "K": 2880, "out": "bf16"},
        # gate/up products of a decode batch: 256 routed rows over 32 experts, HBM bound
        {"name": "grouped_decode", "op": "grouped", "T": 64, "k": 4, "E": 32, "N": 5760, "K": 2880,
         "skew": 0.0, "out": "bf16"},
        # gate/up products of a skewed prefill batch over 128 experts, some of them nearly idle
        {"name": "grouped_skewed_prefill", "op": "grouped", "T": 16384, "k": 4, "E": 128, "N": 5760,
         "K": 2880, "skew": 1.1, "out": "bf16"},
        # weight gradient at ragged sizes: odd token count, widths that fill no tile
        {"name": "weight_grad_odd", "op": "weight_grad", "T": 3001, "k": 1, "E": 8, "M": 712, "N": 1000,
         "skew": 1.0, "out": "fp32"},
        # weight gradient of the down projection in a training step
        {"name": "weight_grad_prefill", "op": "weight_grad", "T": 8192, "k": 4, "E": 32, "M": 2880,
         "N": 2880, "skew": 0.0, "out": "fp32"},
        # input gradient of a tiny layer's gate/up projection: latency of three launches
        {"name": "input_grad_tiny", "op": "input_grad", "T": 16, "k": 4, "E": 8, "N": 512, "K": 256,
         "skew": 0.0, "out": "bf16"},
        # input gradient of the gate/up projection in a training step, weights requantised
        {"name": "input_grad_prefill", "op": "input_grad", "T": 8192, "k": 4, "E": 32, "N": 5760,
         "K": 2880, "skew": 0.0, "out": "bf16"},
        # gradient of the weighted way back: a decode-sized batch, then a prefill batch
        {"name": "combine_backward_decode", "op": "combine_backward", "T": 64, "k": 4, "E": 32,
         "D": 2880, "skew": 0.0},
        {"name": "combine_backward_prefill", "op": "combine_backward", "T": 16384, "k": 4, "E": 128,
         "D": 2880, "skew": 1.1},
        # gradient of the sort: odd token count without, a prefill batch with the router's share
        {"name": "permute_backward_odd", "op": "permute_backward", "T": 1001, "k": 3, "E": 20,
         "D": 320, "skew": 1.0, "router": False},
        {"name": "permute_backward_prefill", "op": "permute_backward", "T": 16384, "k": 4, "E": 128,
         "D": 2880, "skew": 1.1, "router": True},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["matmul", "grouped", "weight_grad", "input_grad", "combine_backward",
                     "permute_backward"])
    out = rng.choice(["bf16", "fp32"])
    if op == "matmul":
        return {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 8, 5760),
                "K": _log(rng, 32, 5760, 32), "out": out}
    E = _log(rng, 1, 128)
    k = rng.randint(1, min(E, 8))
    skew = rng.choice([0.0, 1.1, 2.0])
    if op in ("grouped", "weight_grad", "input_grad"):
        case = {"op": op, "T": _log(rng, 1, 16384 // k), "k": k, "E": E}
        wide = _log(rng, 64, 2880 if E > 32 else 5760, 32)
        if op == "grouped":
            case.update(N=_log(rng, 8, 2880), K=wide)
        elif op == "weight_grad":
            case.update(M=_log(rng, 8, 2880, 8), N=_log(rng, 8, 2880, 8))
        else:
            case.update(N=wide, K=_log(rng, 64, 2880, 8))
        case.update(skew=skew, out=out)
        return case
    case = {"op": op, "T": _log(rng, 1, 65536 // k), "k": k, "E": E, "D": _log(rng, 128, 2880, 64),
            "skew": skew}
    if op == "permute_backward":
        case["router"] = rng.random() < 0.5
    return case


def _rows(c):
    return c["T"] * c["k"]


def work(c):
    mx = 17 / 32  # bytes of one MXFP4 element with its share of the scale
    if c["op"] == "matmul":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": int((M + N) * K * mx + M * N * OUT[c["out"]].itemsize), "flops": 2 * M * N * K}
    S = _rows(c)
    touched = min(c["E"], S)
    if c["op"] == "grouped":
        N, K = c["N"], c["K"]
        return {"bytes": int((S + touched * N) * K * mx + S * N * OUT[c["out"]].itemsize),
                "flops": 2 * S * N * K}
    if c["op"] == "weight_grad":  # bf16 rows of both sides in, one matrix per expert out
        M, N = c["M"], c["N"]
        return {"bytes": S * (M + N) * 2 + c["E"] * M * N * OUT[c["out"]].itemsize,
                "flops": 2 * S * M * N}
    if c["op"] == "input_grad":  # bf16 rows and bf16 weights in
        N, K = c["N"], c["K"]
        return {"bytes": S * N * 2 + touched * N * K * 2 + S * K * OUT[c["out"]].itemsize,
                "flops": 2 * S * N * K}
    T, D = c["T"], c["D"]
    if c["op"] == "combine_backward":
        return {"bytes": T * D * 2 + 2 * S * D * 2 + S * 16, "flops": 3 * S * D}
    router = c["router"]
    return {"bytes": S * D * 2 + T * D * 2 + S * 4 + (S * 8 + c["E"] * D * 2 if router else 0),
            "flops": (3 if router else 1) * S * D}


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, sigma, outliers=0.0):
    x = torch.randn(shape, generator=gen, device=DEV) * sigma
    if outliers:
        x = torch.where(torch.rand(shape, generator=gen, device=DEV) < outliers, x * 20, x)
    return x.to(torch.bfloat16)


def _packed_normal(gen, shape, sigma, outliers=0.0):
    """A normal bf16 tensor [..., K] as MXFP4 codes and scales, one leading index at a time."""
    if len(shape) == 2:
        return _pack(*_quantise(_normal(gen, shape, sigma, outliers).float()))
    parts = [_packed_normal(gen, shape[1:], sigma, outliers) for _ in range(shape[0])]
    return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])


def _routing(gen, c):
    """Expert choice of a batch: indices, weights, the stable order by expert and its inverse."""
    T, k, E = c["T"], c["k"], c["E"]
    logits = torch.randn((T, E), generator=gen, device=DEV)
    rank = torch.arange(1, E + 1, device=DEV, dtype=torch.float32)
    logits = logits - 2 * c["skew"] * rank.log()
    top, idx = logits.topk(k, dim=1)
    flat = idx.reshape(-1)
    order = torch.argsort(flat, stable=True)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(T * k, device=DEV)
    ends = torch.bincount(flat, minlength=E).cumsum(0)
    offsets = torch.cat([ends.new_zeros(1), ends]).to(torch.int32)
    return {"idx": idx.to(torch.int32).contiguous(), "w": torch.softmax(top, 1).contiguous(),
            "pos": pos.to(torch.int32), "offsets": offsets, "bounds": offsets.tolist()}


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    st = {"case": c, "status": torch.zeros(1, dtype=torch.int32, device=DEV)}
    if c["op"] == "matmul":
        st["a"] = _packed_normal(gen, (c["M"], c["K"]), 1.0)
        st["b"] = _packed_normal(gen, (c["N"], c["K"]), 0.02, 0.01)
        st["out"] = torch.empty((c["M"], c["N"]), dtype=OUT[c["out"]], device=DEV)
        return st
    st.update(_routing(gen, c))
    S, E = _rows(c), c["E"]
    if c["op"] == "grouped":
        st["a"] = _packed_normal(gen, (S, c["K"]), 1.0)
        st["b"] = _packed_normal(gen, (E, c["N"], c["K"]), 0.02, 0.01)
        st["out"] = torch.empty((S, c["N"]), dtype=OUT[c["out"]], device=DEV)
    elif c["op"] == "weight_grad":
        st["dy"] = _normal(gen, (S, c["M"]), 0.1)
        st["x"] = _normal(gen, (S, c["N"]), 1.0)
        st["out"] = torch.empty((E, c["M"], c["N"]), dtype=OUT[c["out"]], device=DEV)
        P = (S + 127 * E) // 128 * 128  # every group starts at a multiple of 128
        st["dyq"], st["xq"] = _codes((c["M"], P)), _codes((c["N"], P))
    elif c["op"] == "input_grad":
        st["dy"] = _normal(gen, (S, c["N"]), 0.1)
        st["w"] = torch.stack([_normal(gen, (c["N"], c["K"]), 0.02, 0.01) for _ in range(E)])
        st["out"] = torch.empty((S, c["K"]), dtype=OUT[c["out"]], device=DEV)
        st["dyq"], st["wq"] = _codes((S, c["N"])), _codes((E, c["K"], c["N"]))
    elif c["op"] == "combine_backward":
        st["dout"] = _normal(gen, (c["T"], c["D"]), 0.1)
        st["y"] = _normal(gen, (S, c["D"]), 1.0)
        st["dy"] = torch.empty((S, c["D"]), dtype=torch.bfloat16, device=DEV)
        st["dw"] = torch.empty((c["T"], c["k"]), device=DEV)
        st["dscore"] = torch.empty((c["T"], c["k"]), device=DEV)
    else:
        st["dx_perm"] = _normal(gen, (S, c["D"]), 0.1)
        st["dx"] = torch.empty((c["T"], c["D"]), dtype=torch.bfloat16, device=DEV)
        if c["router"]:
            st["w_router"] = _normal(gen, (E, c["D"]), c["D"] ** -0.5)
            st["dscore"] = torch.randn((c["T"], c["k"]), generator=gen, device=DEV) * 0.1
    return st


def _codes(shape):
    """Buffers of an MXFP4 matrix [..., K]: codes and scales."""
    return (torch.empty(shape[:-1] + (shape[-1] // 2,), dtype=torch.uint8, device=DEV),
            torch.empty(shape[:-1] + (shape[-1] // 32,), dtype=torch.uint8, device=DEV))


# --------------------------------------------------------------- plain form

def _pow2(e):
    """2^e in fp32 from its bits, for integers -127 <= e <= 127."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _quantise(x):
    """fp32 [..., K] -> signed grid values and scale exponents per block of 32."""
    blk = x.unflatten(-1, (-1, 32))
    amax = blk.abs().amax(-1)
    e = (torch.frexp(amax).exponent - 3).clamp(-127, 127)  # floor(log2 amax) - 2
    e = torch.where(amax == 0, -127, e)
    v = blk * _pow2(-e).unsqueeze(-1)
    step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0))
    return ((v / step).round() * step).clamp(-6, 6), e  # ties to the even multiple


def _pack(v, e):
    mag = v.abs()
    code = sum((mag >= g).to(torch.uint8) for g in GRID[1:]) + 8 * torch.signbit(v).to(torch.uint8)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _value(q, s):
    """MXFP4 codes and scales -> fp32."""
    code = torch.stack([q & 15, q >> 4], -1).flatten(-2).int()
    mant, ex = (code & 1).float(), (code >> 1) & 3
    v = torch.where(ex == 0, 0.5 * mant, (1 + 0.5 * mant) * _pow2(ex - 1))
    v = torch.where(code >= 8, -v, v).unflatten(-1, (-1, 32))
    return (v * _pow2(s.int() - 127).unsqueeze(-1)).flatten(-2)


def _rounded(x):
    """The fp32 values that quantising x along its last axis keeps (zeros fill the last block)."""
    K = x.shape[-1]
    x = torch.nn.functional.pad(x.float(), (0, -K % 32))
    v, e = _quantise(x)
    return (v * _pow2(e).unsqueeze(-1)).flatten(-2)[..., :K]


def _plain(st):
    c = st["case"]
    op = c["op"]
    if op == "matmul":
        return (_value(*st["a"]) @ _value(*st["b"]).T).to(OUT[c["out"]])
    b = st["bounds"]
    out = st.get("out")
    if op == "grouped":
        a = _value(*st["a"])
        for e in range(c["E"]):
            if b[e] < b[e + 1]:
                out[b[e]:b[e + 1]] = a[b[e]:b[e + 1]] @ _value(st["b"][0][e], st["b"][1][e]).T
        return out
    if op == "weight_grad":
        for e in range(c["E"]):
            rows = slice(b[e], b[e + 1])
            if b[e] == b[e + 1]:
                out[e] = 0
                continue
            out[e] = _rounded(st["dy"][rows].T) @ _rounded(st["x"][rows].T).T
        return out
    if op == "input_grad":
        dy = _rounded(st["dy"])
        for e in range(c["E"]):
            if b[e] < b[e + 1]:
                out[b[e]:b[e + 1]] = dy[b[e]:b[e + 1]] @ _rounded(st["w"][e].T).T
        return out
    pos = st["pos"].long().view(c["T"], c["k"])
    if op == "combine_backward":
        dout, w = st["dout"].float().unsqueeze(1), st["w"]
        dw = (dout * st["y"][pos].float()).sum(-1)
        dy = torch.empty_like(st["dy"])
        dy[pos] = (w.unsqueeze(-1) * dout).to(torch.bfloat16)
        return {"dy": dy, "dw": dw, "dscore": w * (dw - (w * dw).sum(-1, keepdim=True))}
    dx = st["dx_perm"][pos].float().sum(1)
    if c["router"]:
        dx = dx + (st["dscore"].unsqueeze(-1) * st["w_router"][st["idx"].long()].float()).sum(1)
    return dx.to(torch.bfloat16)


# ------------------------------------------------------------ the library's

def _library(st):
    import mxfp4_quantised_mixture_b200 as moe

    c = st["case"]
    op = c["op"]
    if op == "matmul":
        moe.mxfp4_matmul(*st["a"], *st["b"], st["out"], d_status=st["status"])
        return st["out"]
    if op == "grouped":
        moe.mxfp4_matmul_grouped(*st["a"], st["offsets"], *st["b"], st["out"], d_status=st["status"])
        return st["out"]
    if op == "weight_grad":
        moe.mxfp4_quantize_transposed_grouped(st["dy"], st["offsets"], *st["dyq"],
                                              d_status=st["status"])
        moe.mxfp4_quantize_transposed_grouped(st["x"], st["offsets"], *st["xq"],
                                              d_status=st["status"])
        moe.mxfp4_matmul_grouped_wgrad(*st["dyq"], *st["xq"], st["offsets"], st["out"],
                                       d_status=st["status"])
        return st["out"]
    if op == "input_grad":
        moe.mxfp4_quantize(st["dy"], *st["dyq"], st["status"])
        moe.mxfp4_quantize_transposed(st["w"], *st["wq"], d_status=st["status"])
        moe.mxfp4_matmul_grouped(*st["dyq"], st["offsets"], *st["wq"], st["out"],
                                 d_status=st["status"])
        return st["out"]
    shape = moe.make_shape(c["T"], c["E"], c["k"], c["D"], c["D"])
    if op == "combine_backward":
        moe.moe_combine_backward(st["dout"], st["y"], st["pos"], st["w"], shape, st["dy"], st["dw"],
                                 st["dscore"])
        return {"dy": st["dy"], "dw": st["dw"], "dscore": st["dscore"]}
    if c["router"]:
        moe.moe_permute_backward(st["dx_perm"], st["pos"], shape, st["dx"], st["idx"], st["dscore"],
                                 st["w_router"])
    else:
        moe.moe_permute_backward(st["dx_perm"], st["pos"], shape, st["dx"])
    return st["dx"]


def run(state):
    return _library(state) if own else _plain(state)


# --------------------------------------------------- the definition in 64 bits

def _value64(q, s):
    """Each code's value by the table of the sixteen codes, times its block's power of two."""
    table = torch.tensor(GRID + tuple(-g for g in GRID), dtype=torch.float64, device=q.device)
    out = torch.empty(q.shape[:-1] + (2 * q.shape[-1],), dtype=torch.float64, device=q.device)
    out[..., 0::2], out[..., 1::2] = table[(q % 16).long()], table[(q // 16).long()]
    scale = ((s.long() + 896) << 52).view(torch.float64)  # 2^(s - 127) by its exponent field
    return out * scale.repeat_interleave(32, -1)


def _rounded64(x):
    """Rounding to the block's grid by its thresholds, in 64 bits, along the last axis."""
    x = x.double()
    n = x.shape[-1]
    full = torch.zeros(x.shape[:-1] + (-(-n // 32) * 32,), dtype=torch.float64, device=x.device)
    full[..., :n] = x
    blk = full.reshape(full.shape[:-1] + (-1, 32))
    amax = blk.abs().max(-1, keepdim=True).values
    field = (amax.view(torch.int64) >> 52) - 2  # of the largest magnitude's power of two, over 4
    scale = (field.clamp(min=1023 - 127) << 52).view(torch.float64)
    v = blk.abs() / scale
    # a value between two grid points goes to the upper one past the middle; the middle
    # itself goes to the point whose mantissa bit is 0
    mag = torch.zeros_like(v)
    for lo, hi, up in ((0, .5, False), (.5, 1, True), (1, 1.5, False), (1.5, 2, True), (2, 3, False),
                       (3, 4, True), (4, 6, False)):
        mid = (lo + hi) / 2
        mag = torch.where((v >= mid) if up else (v > mid), float(hi), mag)
    out = torch.where(blk < 0, -mag, mag) * scale
    return out.reshape(full.shape)[..., :n]


def exact(case, seed):
    c = case
    st = prepare(case, seed)
    op = c["op"]
    if op == "matmul":
        return _value64(*st["a"]) @ _value64(*st["b"]).transpose(0, 1)
    b = st["bounds"]
    if op in ("grouped", "input_grad"):
        width = c["N"] if op == "grouped" else c["K"]
        out = torch.zeros((_rows(c), width), dtype=torch.float64, device=DEV)
        for e in range(c["E"]):
            lo, hi = b[e], b[e + 1]
            if hi == lo:
                continue
            if op == "grouped":
                left = _value64(st["a"][0][lo:hi], st["a"][1][lo:hi])
                right = _value64(st["b"][0][e], st["b"][1][e])
            else:
                left = _rounded64(st["dy"][lo:hi])
                right = _rounded64(st["w"][e].transpose(0, 1).contiguous())
            out[lo:hi] = left @ right.transpose(0, 1)
        return out
    if op == "weight_grad":
        out = torch.zeros((c["E"], c["M"], c["N"]), dtype=torch.float64, device=DEV)
        for e in range(c["E"]):
            lo, hi = b[e], b[e + 1]
            if hi > lo:
                out[e] = (_rounded64(st["dy"][lo:hi].transpose(0, 1).contiguous())
                          @ _rounded64(st["x"][lo:hi].transpose(0, 1).contiguous()).transpose(0, 1))
        return out
    # one choice j at a time
    T, k = c["T"], c["k"]
    pos = st["pos"].long().reshape(T, k)
    if op == "combine_backward":
        dout, w = st["dout"].double(), st["w"].double()
        dy = torch.zeros((T * k, c["D"]), dtype=torch.float64, device=DEV)
        dw = torch.zeros((T, k), dtype=torch.float64, device=DEV)
        for j in range(k):
            dy[pos[:, j]] = dout * w[:, j:j + 1]
            dw[:, j] = torch.einsum("td,td->t", dout, st["y"][pos[:, j]].double())
        mean = torch.einsum("tj,tj->t", w, dw)
        return {"dy": dy, "dw": dw, "dscore": w * dw - w * mean[:, None]}
    dx = torch.zeros((T, c["D"]), dtype=torch.float64, device=DEV)
    for j in range(k):
        dx += st["dx_perm"][pos[:, j]].double()
        if c["router"]:
            dx += st["dscore"][:, j:j + 1].double() * st["w_router"][st["idx"][:, j].long()].double()
    return dx
