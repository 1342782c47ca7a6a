"""Thin Python binding of libmoe_mxfp4.so (the MXFP4 Mixture-of-Experts layer
for NVIDIA B200, sm_100a).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  Tensors are torch device tensors (used here for device memory and
streams); their ``data_ptr()`` is handed to the C ABI declared in
``include/moe_mxfp4.h``.  A missing or unloadable library raises at import:
there is no other implementation to fall back to.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_mxfp4.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_SHAPE = 2
MOE_ERR_WORKSPACE = 3
MOE_ERR_UNSUPPORTED = 4
MOE_ERR_CUDA = 5
MOE_ERR_NONFINITE = 6
MOE_ERR_TIMEOUT = 7

WS_PERMUTE, WS_EXPERT_MLP, WS_LAYER = 0, 1, 2
WS_EXPERT_MLP_BLOCK_SCALED, WS_EXPERT_MLP_BF16_DECODE = 3, 4
WS_EXPERT_MLP_UNQUANTISED = 5

# GEMM path of moe_expert_mlp_ex
MOE_MLP_PATH_AUTO = 0
MOE_MLP_PATH_BLOCK_SCALED = 1  # tcgen05 block-scaled MMA on the E2M1 codes
MOE_MLP_PATH_BF16_DECODE = 2   # codes decoded to bf16 into tensor memory

MOE_QUANT_RHT = 1  # random-sign Hadamard transform of each 32-block along K
MOE_QUANT_SR = 2   # stochastic rounding


MOE_OUT_BF16 = 0  # output type of a product
MOE_OUT_FP32 = 1


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {moe_status_string(status)} ({status})")
        self.status = status


class moe_shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32)]

    def __repr__(self):
        return (f"moe_shape(T={self.T}, E={self.E}, k={self.k}, d_model={self.d_model}, "
                f"d_ff={self.d_ff})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python mxfp4_quantised_mixture_b200/build.py`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    st = ctypes.c_int
    lib.mxfp4_quantize.argtypes = [vp, i64, i64, vp, vp, vp, vp]
    lib.mxfp4_quantize.restype = st
    lib.mxfp4_quantize_sr_rht.argtypes = [vp, i64, i64, ctypes.c_uint32, vp, ctypes.c_uint64, vp,
                                          vp, vp, vp]
    lib.mxfp4_quantize_sr_rht.restype = st
    lib.moe_route.argtypes = [vp, i32, i32, i32, vp, vp, vp]
    lib.moe_route.restype = st
    lib.moe_router_topk.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp]
    lib.moe_router_topk.restype = st
    lib.moe_permute.argtypes = [vp, vp, moe_shape, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_permute.restype = st
    lib.moe_expert_mlp.argtypes = [vp, vp, moe_shape, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_expert_mlp.restype = st
    lib.moe_expert_mlp_ex.argtypes = [vp, vp, moe_shape, vp, vp, vp, vp, vp, vp, vp, sz, i32, i32,
                                      vp]
    lib.moe_expert_mlp_ex.restype = st
    lib.moe_expert_mlp_unquantised.argtypes = [vp, vp, moe_shape, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_expert_mlp_unquantised.restype = st
    lib.moe_combine.argtypes = [vp, vp, vp, moe_shape, vp, vp]
    lib.moe_combine.restype = st
    f32 = ctypes.c_float
    lib.mxfp4_transposed_width.argtypes = [i64, i32]
    lib.mxfp4_transposed_width.restype = i64
    lib.mxfp4_quantize_transposed.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp]
    lib.mxfp4_quantize_transposed.restype = st
    lib.mxfp4_quantize_transposed_grouped.argtypes = [vp, i64, i64, vp, i32, vp, vp, vp, vp]
    lib.mxfp4_quantize_transposed_grouped.restype = st
    lib.mxfp4_matmul.argtypes = [vp, vp, vp, vp, i64, i64, i64, f32, vp, i32, vp, vp]
    lib.mxfp4_matmul.restype = st
    lib.mxfp4_matmul_ex.argtypes = [vp, vp, vp, vp, i64, i64, i64, f32, vp, i32, vp, i32, vp]
    lib.mxfp4_matmul_ex.restype = st
    lib.mxfp4_matmul_grouped.argtypes = [vp, vp, vp, i32, vp, vp, i64, i64, i64, f32, vp, i32, vp,
                                         vp]
    lib.mxfp4_matmul_grouped.restype = st
    lib.mxfp4_matmul_grouped_wgrad.argtypes = [vp, vp, vp, vp, vp, i32, i64, i64, i64, f32, vp, i32,
                                               vp, vp]
    lib.mxfp4_matmul_grouped_wgrad.restype = st
    lib.moe_combine_backward.argtypes = [vp, vp, vp, vp, moe_shape, vp, vp, vp, vp]
    lib.moe_combine_backward.restype = st
    lib.moe_permute_backward.argtypes = [vp, vp, moe_shape, vp, vp, vp, vp, vp]
    lib.moe_permute_backward.restype = st
    lib.moe_layer_forward.argtypes = [vp, vp, moe_shape, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_layer_forward.restype = st
    lib.moe_layer_forward_static.argtypes = [vp, vp, moe_shape, vp, vp, vp, vp, vp, vp]
    lib.moe_layer_forward_static.restype = st
    lib.moe_layer_static_status.argtypes = [vp, vp]
    lib.moe_layer_static_status.restype = st
    lib.moe_workspace_size.argtypes = [moe_shape, ctypes.c_int]
    lib.moe_workspace_size.restype = sz
    lib.moe_status_string.argtypes = [st]
    lib.moe_status_string.restype = ctypes.c_char_p
    return lib


lib = _load()


def _p(t) -> int | None:
    """Device pointer of a tensor argument (None and raw integer addresses
    pass through).  The C ABI reads dense row-major device arrays, so a
    strided view or a host tensor is refused here rather than misread."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("tensor arguments must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous (dense row-major)")
    return t.data_ptr()


def _s(stream) -> int | None:
    if stream is None:
        import torch

        # the current device's current stream, without building a Stream object
        # (0.4 us instead of 3.2) where this torch has the lookup
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return raw(torch.cuda.current_device()) if raw else torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _check(fn: str, status: int) -> None:
    if status != MOE_OK:
        raise MoeError(fn, status)


def make_shape(T: int, E: int, k: int, d_model: int, d_ff: int) -> moe_shape:
    return moe_shape(T, E, k, d_model, d_ff)


def moe_status_string(status: int) -> str:
    return lib.moe_status_string(int(status)).decode()


def moe_workspace_size(shape: moe_shape, which: int) -> int:
    return int(lib.moe_workspace_size(shape, which))


def mxfp4_quantize(w_bf16, q_packed, scales, d_status=None, stream=None) -> None:
    """w_bf16 [rows][K] bf16 -> q_packed [rows][K/2] u8, scales [rows][K/32] u8."""
    K = w_bf16.shape[-1]
    rows = w_bf16.numel() // K if K else 0
    _check("mxfp4_quantize", lib.mxfp4_quantize(_p(w_bf16), rows, K, _p(q_packed), _p(scales),
                                                _p(d_status), _s(stream)))


def mxfp4_quantize_sr_rht(w_bf16, flags: int, rht_signs, seed: int, q_packed, scales,
                          d_status=None, stream=None) -> None:
    """w_bf16 [rows][K] bf16 -> q_packed [rows][K/2] u8, scales [rows][K/32] u8,
    with the optional transform (MOE_QUANT_RHT; rht_signs [K/32] int32/uint32)
    and stochastic rounding (MOE_QUANT_SR, Philox keyed by ``seed``)."""
    K = w_bf16.shape[-1]
    rows = w_bf16.numel() // K if K else 0
    _check("mxfp4_quantize_sr_rht",
           lib.mxfp4_quantize_sr_rht(_p(w_bf16), rows, K, int(flags) & 0xFFFFFFFF, _p(rht_signs),
                                     int(seed) & 0xFFFFFFFFFFFFFFFF, _p(q_packed), _p(scales),
                                     _p(d_status), _s(stream)))


_types: tuple = ()  # (uint8, int32, float32, the 16-bit types that carry bf16), once torch is there


def _dtypes() -> tuple:
    global _types
    if not _types:
        import torch

        _types = ((torch.uint8,), (torch.int32,), (torch.float32,),
                  (torch.bfloat16, torch.int16, torch.uint16))
    return _types


def _args(fn: str, *specs) -> list:
    """Device pointers of a call's tensors, given as (tensor, shape, types); a
    tensor that is None passes through.  Shapes or types that contradict one
    another are refused (the C call would read or write past the smaller one),
    and so are tensors off the current device, whose stream runs the call, and
    strided views."""
    import torch

    dev = torch.cuda.current_device() if torch.cuda.is_initialized() else None
    out, off = [], False
    for t, shape, types in specs:
        if t is None:
            out.append(None)
            continue
        if (shape is not None and t.shape != shape) or t.dtype not in types:
            raise ValueError(f"{fn}: the tensors' shapes or types do not belong together")
        if t.get_device() != dev:
            off = True
        if not t.is_contiguous():
            raise ValueError(f"{fn}: tensor arguments must be contiguous (dense row-major)")
        out.append(t.data_ptr())
    if off:
        raise ValueError(f"{fn}: tensor arguments must live on a CUDA device, the current one")
    return out


def _out_type(fn: str, out) -> int:
    import torch

    if out.dtype is torch.bfloat16:
        return MOE_OUT_BF16
    if out.dtype is torch.float32:
        return MOE_OUT_FP32
    raise ValueError(f"{fn}: the output is bfloat16 or float32, not {out.dtype}")


def mxfp4_transposed_width(rows: int, E: int = 0) -> int:
    """Positions along the contraction axis of a transposed MXFP4 matrix: rows
    rounded up to 32, or, with E groups of rows, room for each of them to start
    at a multiple of 128."""
    return int(lib.mxfp4_transposed_width(int(rows), int(E)))


def mxfp4_quantize_transposed(w_bf16, q_packed, scales, d_status=None, stream=None) -> None:
    """w_bf16 [..., R, C] bf16 -> q_packed [..., C, P/2] u8, scales [..., C, P/32] u8,
    P = mxfp4_transposed_width(R): mxfp4_quantize of the transpose."""
    fn, (u8, i32, _, b16) = "mxfp4_quantize_transposed", _dtypes()
    shape = tuple(w_bf16.shape)
    R, C = shape[-2:]
    P, lead = mxfp4_transposed_width(R), shape[:-2] + (C,)
    w, q, sc, st = _args(fn, (w_bf16, shape, b16), (q_packed, lead + (P // 2,), u8),
                         (scales, lead + (P // 32,), u8), (d_status, None, i32))
    batch = w_bf16.numel() // (R * C) if R * C else 0
    _check(fn, lib.mxfp4_quantize_transposed(w, batch, R, C, q, sc, st, _s(stream)))


def mxfp4_quantize_transposed_grouped(w_bf16, offsets, q_packed, scales, d_status=None,
                                      stream=None) -> None:
    """w_bf16 [S, C] bf16, offsets [E+1] i32 -> q_packed [C, P/2], scales [C, P/32],
    P = mxfp4_transposed_width(S, E), every group at a multiple of 128 positions."""
    fn, (u8, i32, _, b16) = "mxfp4_quantize_transposed_grouped", _dtypes()
    S, C = w_bf16.shape
    E = offsets.numel() - 1
    P = mxfp4_transposed_width(S, E)
    w, off, q, sc, st = _args(fn, (w_bf16, (S, C), b16), (offsets, (E + 1,), i32),
                              (q_packed, (C, P // 2), u8), (scales, (C, P // 32), u8),
                              (d_status, None, i32))
    _check(fn, lib.mxfp4_quantize_transposed_grouped(w, S, C, off, E, q, sc, st, _s(stream)))


def _matmul_args(fn: str, a_q, a_s, b_q, b_s, out, alpha: float, d_status) -> tuple:
    u8, i32, _, _ = _dtypes()
    (M, N), h, kind = out.shape, a_q.shape[-1], _out_type(fn, out)
    aq, sa, bq, sb, o, st = _args(fn, (a_q, (M, h), u8), (a_s, (M, h // 16), u8), (b_q, (N, h), u8),
                                  (b_s, (N, h // 16), u8), (out, (M, N), (out.dtype,)),
                                  (d_status, None, i32))
    return aq, sa, bq, sb, M, N, 2 * h, float(alpha), o, kind, st


def mxfp4_matmul(a_q, a_s, b_q, b_s, out, alpha: float = 1.0, d_status=None, stream=None) -> None:
    """out [M, N] (bf16 or fp32) = alpha * A B^T of MXFP4 A [M, K] and B [N, K]."""
    fn = "mxfp4_matmul"
    args = _matmul_args(fn, a_q, a_s, b_q, b_s, out, alpha, d_status)
    _check(fn, lib.mxfp4_matmul(*args, _s(stream)))


def mxfp4_matmul_ex(a_q, a_s, b_q, b_s, out, alpha: float = 1.0, d_status=None,
                    test_timeout_cta: int = -1, stream=None) -> None:
    """mxfp4_matmul; test_timeout_cta >= 0 is testing support (see the C header)."""
    fn = "mxfp4_matmul_ex"
    args = _matmul_args(fn, a_q, a_s, b_q, b_s, out, alpha, d_status)
    _check(fn, lib.mxfp4_matmul_ex(*args, int(test_timeout_cta), _s(stream)))


def mxfp4_matmul_grouped(a_q, a_s, offsets, b_q, b_s, out, alpha: float = 1.0, d_status=None,
                         stream=None) -> None:
    """out [S, N] = alpha * (rows of group e of A [S, K]) B_e^T, B [E, N, K], groups by
    offsets [E+1]; rows in no group are left as they were."""
    fn, (u8, i32, _, _) = "mxfp4_matmul_grouped", _dtypes()
    (S, N), h, kind, E = out.shape, a_q.shape[-1], _out_type(fn, out), offsets.numel() - 1
    aq, sa, off, bq, sb, o, st = _args(fn, (a_q, (S, h), u8), (a_s, (S, h // 16), u8),
                                       (offsets, (E + 1,), i32), (b_q, (E, N, h), u8),
                                       (b_s, (E, N, h // 16), u8), (out, (S, N), (out.dtype,)),
                                       (d_status, None, i32))
    _check(fn, lib.mxfp4_matmul_grouped(aq, sa, off, E, bq, sb, S, N, 2 * h, float(alpha), o, kind, st,
                                        _s(stream)))


def mxfp4_matmul_grouped_wgrad(a_q, a_s, b_q, b_s, offsets, out, alpha: float = 1.0, d_status=None,
                               stream=None) -> None:
    """out [E, M, N] = alpha * A_e B_e^T over the positions of group e of A [M, P] and
    B [N, P] (mxfp4_quantize_transposed_grouped's outputs for the same offsets)."""
    fn, (u8, i32, _, _) = "mxfp4_matmul_grouped_wgrad", _dtypes()
    (E, M, N), h, kind = out.shape, a_q.shape[-1], _out_type(fn, out)
    aq, sa, bq, sb, off, o, st = _args(fn, (a_q, (M, h), u8), (a_s, (M, h // 16), u8), (b_q, (N, h), u8),
                                       (b_s, (N, h // 16), u8), (offsets, (E + 1,), i32),
                                       (out, (E, M, N), (out.dtype,)), (d_status, None, i32))
    _check(fn, lib.mxfp4_matmul_grouped_wgrad(aq, sa, bq, sb, off, E, M, N, 2 * h, float(alpha), o, kind,
                                              st, _s(stream)))


def moe_route(logits, k: int, topk_idx, topk_w, stream=None) -> None:
    T, E = logits.shape
    _check("moe_route", lib.moe_route(_p(logits), T, E, k, _p(topk_idx), _p(topk_w), _s(stream)))


def moe_router_topk(x, w_router, k: int, topk_idx, topk_w, logits=None, d_status=None,
                    stream=None) -> None:
    """x [T][D] bf16, w_router [E][D] bf16 -> topk_idx [T][k] i32, topk_w [T][k] f32
    (and logits [T][E] f32 when given)."""
    T, D = x.shape
    E = w_router.shape[0]
    _check("moe_router_topk", lib.moe_router_topk(_p(x), _p(w_router), T, D, E, k, _p(logits),
                                                  _p(topk_idx), _p(topk_w), _p(d_status),
                                                  _s(stream)))


def moe_permute(topk_idx, x, shape: moe_shape, counts, offsets, sorted_slot, slot_pos, x_perm,
                ws=None, stream=None) -> None:
    _check("moe_permute", lib.moe_permute(_p(topk_idx), _p(x), shape, _p(counts), _p(offsets),
                                          _p(sorted_slot), _p(slot_pos), _p(x_perm), _p(ws),
                                          _nbytes(ws), _s(stream)))


def moe_expert_mlp(x_perm, offsets, shape: moe_shape, wgu_q, wgu_s, wdn_q, wdn_s, h, y_perm, ws,
                   stream=None) -> None:
    _check("moe_expert_mlp", lib.moe_expert_mlp(_p(x_perm), _p(offsets), shape, _p(wgu_q),
                                                _p(wgu_s), _p(wdn_q), _p(wdn_s), _p(h), _p(y_perm),
                                                _p(ws), _nbytes(ws), _s(stream)))


def moe_expert_mlp_ex(x_perm, offsets, shape: moe_shape, wgu_q, wgu_s, wdn_q, wdn_s, h, y_perm, ws,
                      path: int = MOE_MLP_PATH_AUTO, test_timeout_cta: int = -1,
                      stream=None) -> None:
    """moe_expert_mlp on a chosen GEMM path (MOE_MLP_PATH_*); ws sized by
    moe_workspace_size(shape, WS_EXPERT_MLP / _BLOCK_SCALED / _BF16_DECODE).
    test_timeout_cta >= 0 is testing support (see the C header)."""
    _check("moe_expert_mlp_ex",
           lib.moe_expert_mlp_ex(_p(x_perm), _p(offsets), shape, _p(wgu_q), _p(wgu_s), _p(wdn_q),
                                 _p(wdn_s), _p(h), _p(y_perm), _p(ws), _nbytes(ws), int(path),
                                 int(test_timeout_cta), _s(stream)))


def moe_expert_mlp_unquantised(x_perm, offsets, shape: moe_shape, w_gu, w_dn, h, y_perm, ws,
                               stream=None) -> None:
    """The grouped expert MLP on unquantised bf16 weights w_gu [E][2F][D] and
    w_dn [E][D][F]; ws sized by moe_workspace_size(shape, WS_EXPERT_MLP_UNQUANTISED)."""
    _check("moe_expert_mlp_unquantised",
           lib.moe_expert_mlp_unquantised(_p(x_perm), _p(offsets), shape, _p(w_gu), _p(w_dn),
                                          _p(h), _p(y_perm), _p(ws), _nbytes(ws), _s(stream)))


def moe_combine(y_perm, slot_pos, topk_w, shape: moe_shape, out, stream=None) -> None:
    _check("moe_combine", lib.moe_combine(_p(y_perm), _p(slot_pos), _p(topk_w), shape, _p(out),
                                          _s(stream)))


def moe_combine_backward(dout, y_perm, slot_pos, topk_w, shape: moe_shape, dy_perm, dtopk_w=None,
                         dscore=None, stream=None) -> None:
    """Gradients of moe_combine: dy_perm [S][D], dtopk_w [T][k], and dscore [T][k] of the
    k chosen logits through the softmax (the last two when given)."""
    fn, (_, i32, f32, b16) = "moe_combine_backward", _dtypes()
    T, k, D = shape.T, shape.k, shape.d_model
    rows, per = (T * k, D), (T, k)
    slots = (T * k,) if slot_pos.ndim == 1 else per
    g, y, pos, w, dy, dw, ds = _args(fn, (dout, (T, D), b16), (y_perm, rows, b16), (slot_pos, slots, i32),
                                     (topk_w, per, f32), (dy_perm, rows, b16), (dtopk_w, per, f32),
                                     (dscore, per, f32))
    _check(fn, lib.moe_combine_backward(g, y, pos, w, shape, dy, dw, ds, _s(stream)))


def moe_permute_backward(dx_perm, slot_pos, shape: moe_shape, dx, topk_idx=None, dscore=None,
                         w_router=None, stream=None) -> None:
    """Gradient of moe_permute's gather: dx [T][D], plus the router's share when
    topk_idx [T][k], dscore [T][k] and w_router [E][D] are given."""
    fn, (_, i32, f32, b16) = "moe_permute_backward", _dtypes()
    T, k, D = shape.T, shape.k, shape.d_model
    slots = (T * k,) if slot_pos.ndim == 1 else (T, k)
    g, pos, o, idx, ds, wr = _args(fn, (dx_perm, (T * k, D), b16), (slot_pos, slots, i32),
                                   (dx, (T, D), b16), (topk_idx, (T, k), i32), (dscore, (T, k), f32),
                                   (w_router, (shape.E, D), b16))
    _check(fn, lib.moe_permute_backward(g, pos, shape, o, idx, ds, wr, _s(stream)))


def moe_layer_forward(x, logits, shape: moe_shape, wgu_q, wgu_s, wdn_q, wdn_s, out, ws,
                      stream=None) -> None:
    _check("moe_layer_forward", lib.moe_layer_forward(_p(x), _p(logits), shape, _p(wgu_q),
                                                      _p(wgu_s), _p(wdn_q), _p(wdn_s), _p(out),
                                                      _p(ws), _nbytes(ws), _s(stream)))


STATIC_SCRATCH_BYTES = 16 << 20


def moe_layer_forward_static(x, logits, shape: moe_shape, wgu_q, wgu_s, wdn_q, wdn_s, out,
                             stream=None) -> None:
    """moe_layer_forward with the intermediates in the library's own 16 MiB
    device array (for callers that cannot allocate); see the C header."""
    _check("moe_layer_forward_static",
           lib.moe_layer_forward_static(_p(x), _p(logits), shape, _p(wgu_q), _p(wgu_s), _p(wdn_q),
                                        _p(wdn_s), _p(out), _s(stream)))


def moe_layer_static_status(d_status, stream=None) -> None:
    """Copy the device status word of the last moe_layer_forward_static call
    on this device into d_status (a device int32 tensor), on the stream."""
    _check("moe_layer_static_status", lib.moe_layer_static_status(_p(d_status), _s(stream)))


def alloc_workspace(shape: moe_shape, which: int, device="cuda"):
    """A device byte tensor of moe_workspace_size(shape, which) bytes (at least 256)."""
    import torch

    n = max(256, moe_workspace_size(shape, which))
    return torch.empty(n, dtype=torch.uint8, device=device)


__all__ = ["moe_shape", "make_shape", "MoeError", "mxfp4_quantize", "mxfp4_quantize_sr_rht",
           "MOE_QUANT_RHT", "MOE_QUANT_SR",
           "mxfp4_transposed_width", "mxfp4_quantize_transposed",
           "mxfp4_quantize_transposed_grouped", "mxfp4_matmul", "mxfp4_matmul_ex",
           "mxfp4_matmul_grouped", "mxfp4_matmul_grouped_wgrad", "MOE_OUT_BF16", "MOE_OUT_FP32",
           "moe_combine_backward", "moe_permute_backward", "moe_route",
           "moe_router_topk", "moe_permute",
           "moe_expert_mlp", "moe_expert_mlp_ex", "moe_expert_mlp_unquantised", "moe_combine", "moe_layer_forward",
           "moe_layer_forward_static", "moe_layer_static_status",
           "moe_workspace_size",
           "moe_status_string", "alloc_workspace", "lib", "LIB_PATH"]
