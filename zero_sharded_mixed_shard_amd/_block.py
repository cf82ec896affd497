"""ctypes binding of the operators around a block's linear layers (see
include/zero_shard_block.h for the contract)."""
from __future__ import annotations

import ctypes

import torch

from ._binding import _FORMATS, _f32, _i32, _u64, _vp, lib
from ._grad import (_F32, _U8, _call, _flat, _matrix, _refuse, _workspace, _workspace_bytes,
                    ACT_BLOCK)

BLOCK = 128                                     # ZERO_BLOCK
NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2       # zero_norm


class _Residual(ctypes.Structure):              # zero_residual
    _fields_ = [("rows", _u64), ("cols", _u64), ("dt", _i32), ("res_dt", _i32), ("post", _i32),
                ("pre", _i32), ("post_weight", _vp), ("post_bias", _vp), ("gate", _vp),
                ("pre_weight", _vp), ("pre_bias", _vp), ("eps", _f32), ("res_scale", _f32),
                ("p", _f32), ("seed", _u64), ("offset", _u64), ("d_offset", _vp)]


class _ResidualGrads(ctypes.Structure):         # zero_residual_grads
    _fields_ = [("post_weight", _vp), ("post_bias", _vp), ("gate", _vp), ("pre_weight", _vp),
                ("pre_bias", _vp)]


_block_p, _grads_p = ctypes.POINTER(_Residual), ctypes.POINTER(_ResidualGrads)
lib.zero_block_quant.argtypes = [_vp, _vp, _vp, _vp, _vp, _u64, _i32, _i32, _u64, _u64, _vp]
lib.zero_block_load.argtypes = [_vp, _u64, _i32, _vp, _vp, _i32, _u64, _u64, _vp]
lib.zero_block_product.argtypes = [_vp, _u64, _i32, _vp, _vp, ctypes.c_uint32, _vp, _vp, _u64,
                                   _u64, _u64, _vp, _u64, _vp]
lib.zero_block_product_workspace.argtypes = [_u64, _u64, _u64, ctypes.POINTER(ctypes.c_uint64)]
lib.zero_dropout.argtypes = [_vp, _u64, _vp, _u64, _i32, _u64, _u64, _f32, _u64, _u64, _vp, _vp]
lib.zero_residual_norm.argtypes = [_vp, _u64, _vp, _u64, _vp, _vp, _u64, _vp, _u64, _block_p, _vp]
lib.zero_residual_norm_backward.argtypes = [
    _vp, _u64, _vp, _u64, _grads_p, _i32, ctypes.c_int32, _vp, _u64, _vp, _u64, _vp, _u64, _vp,
    _u64, _vp, _block_p, _vp, _u64, _vp]
lib.zero_residual_norm_workspace.argtypes = [_u64, _u64, ctypes.POINTER(ctypes.c_uint64)]
for _f in ("zero_block_quant", "zero_block_load", "zero_block_product",
           "zero_block_product_workspace", "zero_dropout", "zero_residual_norm",
           "zero_residual_norm_backward", "zero_residual_norm_workspace"):
    getattr(lib, _f).restype = _i32


# ---- matrices in 8 bits with one power of two for each block of 128 ----------------------

def _blocks(n: int) -> int:
    return -(-n // BLOCK)


def _codes(q, e, square: bool, dev, q_name: str = "q", e_name: str = "e") -> tuple:
    """(q pointer, e pointer, shape) of a coded matrix."""
    if not (isinstance(q, torch.Tensor) and q.dim() == 2):
        _refuse(q, q_name, _U8, dev, "a matrix of shape (rows, cols)")
    rows, cols = q.shape
    return (_flat(q, q_name, _U8, (rows, cols), dev),
            _flat(e, e_name, _U8, (_blocks(rows) if square else rows, _blocks(cols)), dev),
            q.shape)


def zero_block_quant(q: torch.Tensor, e: torch.Tensor, x: torch.Tensor, square: bool = False,
                     qt: torch.Tensor | None = None, et: torch.Tensor | None = None,
                     stream=None) -> None:
    """Codes q[rows, cols] and exponents e of x, uint8: e[rows, ceil(cols/128)], or with
    square blocks e[ceil(rows/128), ceil(cols/128)] and, if given, the transposed codes
    qt[cols, rows] with their exponents et."""
    p_x, ldx = _matrix(x, "x", _FORMATS)
    dev, shape = x.get_device(), x.shape
    p_q, p_e, held = _codes(q, e, square, dev)
    if held != shape:
        raise ValueError(f"q must have x's shape {tuple(shape)}, got {tuple(held)}")
    if (qt is None) != (et is None):
        raise ValueError("qt and et go together")
    if qt is not None and not square:
        raise ValueError("transposed codes need square blocks")
    p_qt = p_et = None
    if qt is not None:
        p_qt, p_et, turned = _codes(qt, et, True, dev, "qt", "et")
        if tuple(turned) != (shape[1], shape[0]):
            raise ValueError(f"qt must have shape {(shape[1], shape[0])}, got {tuple(turned)}")
    _call("zero_block_quant", lib.zero_block_quant, dev, stream, p_q, p_e, p_qt, p_et, p_x, ldx,
          _FORMATS[x.dtype], int(bool(square)), shape[0], shape[1])


def zero_block_load(x: torch.Tensor, q: torch.Tensor, e: torch.Tensor, square: bool = False,
                    stream=None) -> None:
    """x = the values the codes (q, e) stand for."""
    p_x, ldx = _matrix(x, "x", _FORMATS)
    dev = x.get_device()
    p_q, p_e, shape = _codes(q, e, square, dev)
    if x.shape != shape:
        raise ValueError(f"x must have q's shape {tuple(shape)}, got {tuple(x.shape)}")
    _call("zero_block_load", lib.zero_block_load, dev, stream, p_x, ldx, _FORMATS[x.dtype], p_q,
          p_e, int(bool(square)), shape[0], shape[1])


def zero_block_product_workspace(m: int, n: int, k: int) -> int:
    """Bytes of workspace zero_block_product needs for these extents."""
    return _workspace_bytes("zero_block_product_workspace", m, n, k)


def zero_block_product(y: torch.Tensor, qa: torch.Tensor, ea: torch.Tensor, qb: torch.Tensor,
                       eb: torch.Tensor, workspace: torch.Tensor | None = None,
                       stream=None) -> None:
    """y[m, n] = a b^T of two coded matrices: a[m, k] with ea[m, ceil(k/128)], or a
    checkpoint with ea[m, ceil(k/32)]; b[n, k] in square blocks."""
    p_y, ldy = _matrix(y, "y", _FORMATS)
    dev, (m, n) = y.get_device(), y.shape
    p_b, p_eb, (n_b, k) = _codes(qb, eb, True, dev, "qb", "eb")
    if n_b != n:
        raise ValueError(f"qb holds {n_b} rows, y {n} columns")
    p_a = _flat(qa, "qa", _U8, (m, k), dev)
    wide = (m, _blocks(k))
    a_block = BLOCK if isinstance(ea, torch.Tensor) and ea.shape == wide else ACT_BLOCK
    p_ea = _flat(ea, "ea", _U8, wide if a_block == BLOCK else (m, -(-k // ACT_BLOCK)), dev)
    p_ws, n_ws = _workspace(workspace, dev)
    _call("zero_block_product", lib.zero_block_product, dev, stream, p_y, ldy, _FORMATS[y.dtype],
          p_a, p_ea, a_block, p_b, p_eb, m, n, k, p_ws, n_ws)


# ---- dropout -----------------------------------------------------------------------------

_I64 = (torch.int64,)


def zero_dropout(y: torch.Tensor, x: torch.Tensor, p: float, seed: int, offset: int = 0,
                 d_offset: torch.Tensor | None = None, stream=None) -> None:
    """y = x with the mask of (seed, offset) applied; the same call with dy for x is the
    backward pass.  d_offset: one int64 on the device, added to offset.  y may be x."""
    p_x, ldx = _matrix(x, "x", _FORMATS)
    dev, shape = x.get_device(), x.shape
    p_y, ldy = _matrix(y, "y", (x.dtype,), shape, dev)
    p_o = None if d_offset is None else _flat(d_offset, "d_offset", _I64, (1,), dev)
    _call("zero_dropout", lib.zero_dropout, dev, stream, p_y, ldy, p_x, ldx, _FORMATS[x.dtype],
          shape[0], shape[1], p, seed, offset, p_o)


# ---- the step between two blocks -----------------------------------------------------------

def _description(shape, dt, res_dt, dev, post, pre, post_weight, post_bias, gate, pre_weight,
                 pre_bias, eps, res_scale, p, seed, offset, d_offset) -> _Residual:
    # (spelled out: this runs on every call)
    dts, vec = (dt,), shape[1:]
    return _Residual(
        shape[0], shape[1], _FORMATS[dt], _FORMATS[res_dt], post, pre,
        None if post_weight is None else _flat(post_weight, "post_weight", dts, vec, dev),
        None if post_bias is None else _flat(post_bias, "post_bias", dts, vec, dev),
        None if gate is None else _flat(gate, "gate", dts, vec, dev),
        None if pre_weight is None else _flat(pre_weight, "pre_weight", dts, vec, dev),
        None if pre_bias is None else _flat(pre_bias, "pre_bias", dts, vec, dev),
        eps, res_scale, p, seed, offset,
        None if d_offset is None else _flat(d_offset, "d_offset", _I64, (1,), dev))


def _pointer(t, name: str, dtypes, shape, dev) -> tuple:
    return (None, 0) if t is None else _matrix(t, name, dtypes, shape, dev)


def zero_residual_norm(u: torch.Tensor | None, h: torch.Tensor | None,
                       stats: torch.Tensor | None, r: torch.Tensor, f: torch.Tensor | None = None,
                       *, post: int = NORM_NONE, pre: int = NORM_RMS,
                       post_weight: torch.Tensor | None = None,
                       post_bias: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                       pre_weight: torch.Tensor | None = None,
                       pre_bias: torch.Tensor | None = None, eps: float = 1e-5,
                       res_scale: float = 1.0, p: float = 0.0, seed: int = 0, offset: int = 0,
                       d_offset: torch.Tensor | None = None, stream=None) -> None:
    """u = res_scale r + gate drop(post(f)) and h = pre(u), with the rows' statistics in
    stats[rows, 4]; without f (and u) h = pre(r).  u may be r."""
    p_r, ldr = _matrix(r, "r", _FORMATS)
    dev, shape, res_dt = r.get_device(), r.shape, r.dtype
    kind = f if f is not None else h
    if not isinstance(kind, torch.Tensor):
        raise TypeError("f or h must be a torch.Tensor")
    dt = kind.dtype
    if dt not in _FORMATS:
        _refuse(kind, "f" if f is not None else "h", _FORMATS, dev, "a matrix")
    p_f, ldf = _pointer(f, "f", (dt,), shape, dev)
    p_h, ldh = _pointer(h, "h", (dt,), shape, dev)
    p_u, ldu = _pointer(u, "u", (res_dt,), shape, dev)
    p_s = None if stats is None else _flat(stats, "stats", _F32, (shape[0], 4), dev)
    block = _description(shape, dt, res_dt, dev, post, pre, post_weight, post_bias, gate,
                         pre_weight, pre_bias, eps, res_scale, p, seed, offset, d_offset)
    _call("zero_residual_norm", lib.zero_residual_norm, dev, stream, p_u, ldu, p_h, ldh, p_s, p_r,
          ldr, p_f, ldf, ctypes.byref(block))


def zero_residual_norm_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace zero_residual_norm_backward needs for these extents."""
    return _workspace_bytes("zero_residual_norm_workspace", rows, cols)


def zero_residual_norm_backward(df: torch.Tensor | None, dr: torch.Tensor,
                                dh: torch.Tensor | None, du: torch.Tensor | None,
                                f: torch.Tensor | None, u: torch.Tensor, stats: torch.Tensor, *,
                                post: int = NORM_NONE, pre: int = NORM_RMS,
                                post_weight: torch.Tensor | None = None,
                                post_bias: torch.Tensor | None = None,
                                gate: torch.Tensor | None = None,
                                pre_weight: torch.Tensor | None = None,
                                pre_bias: torch.Tensor | None = None, eps: float = 1e-5,
                                res_scale: float = 1.0, p: float = 0.0, seed: int = 0,
                                offset: int = 0, d_offset: torch.Tensor | None = None,
                                d_post_weight: torch.Tensor | None = None,
                                d_post_bias: torch.Tensor | None = None,
                                d_gate: torch.Tensor | None = None,
                                d_pre_weight: torch.Tensor | None = None,
                                d_pre_bias: torch.Tensor | None = None, first: bool = True,
                                workspace: torch.Tensor | None = None, stream=None) -> None:
    """Gradients of zero_residual_norm: df, dr and those of the parameters that are asked
    for, all of one format (stored, or FP32 and not first: added).  df may be dh, dr may
    be du."""
    p_u, ldu = _matrix(u, "u", _FORMATS)
    dev, shape, res_dt = u.get_device(), u.shape, u.dtype
    kind = f if f is not None else dh
    if not isinstance(kind, torch.Tensor):
        raise TypeError("f or dh must be a torch.Tensor")
    dt = kind.dtype
    if dt not in _FORMATS:
        _refuse(kind, "f" if f is not None else "dh", _FORMATS, dev, "a matrix")
    p_f, ldf = _pointer(f, "f", (dt,), shape, dev)
    p_df, lddf = _pointer(df, "df", (dt,), shape, dev)
    p_dh, lddh = _pointer(dh, "dh", (dt,), shape, dev)
    p_du, lddu = _pointer(du, "du", (res_dt,), shape, dev)
    p_dr, lddr = _matrix(dr, "dr", (res_dt,), shape, dev)
    p_s = _flat(stats, "stats", _F32, (shape[0], 4), dev)
    block = _description(shape, dt, res_dt, dev, post, pre, post_weight, post_bias, gate,
                         pre_weight, pre_bias, eps, res_scale, p, seed, offset, d_offset)
    named = (("d_post_weight", d_post_weight), ("d_post_bias", d_post_bias), ("d_gate", d_gate),
             ("d_pre_weight", d_pre_weight), ("d_pre_bias", d_pre_bias))
    grad_dt, grads = dt, []
    for _, t in named:
        if isinstance(t, torch.Tensor) and t.dtype == torch.float32:
            grad_dt = torch.float32
    for name, t in named:
        grads.append(None if t is None else _flat(t, name, (grad_dt,), shape[1:], dev))
    p_ws, n_ws = _workspace(workspace, dev)
    _call("zero_residual_norm_backward", lib.zero_residual_norm_backward, dev, stream, p_df, lddf,
          p_dr, lddr, ctypes.byref(_ResidualGrads(*grads)), _FORMATS[grad_dt], int(bool(first)),
          p_dh, lddh, p_du, lddu, p_f, ldf, p_u, ldu, p_s, ctypes.byref(block), p_ws, n_ws)
