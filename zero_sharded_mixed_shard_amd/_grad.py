"""ctypes binding of the gradient operators (see include/zero_shard_grad.h for the contract)."""
from __future__ import annotations

import ctypes

import torch

from ._binding import (_DTYPES, _FORMATS, _ctl_ptr, _f32, _i32, _raw_current_stream,
                       _stream_handle, _u64, _vp, ZeroError, lib)

ACT_BLOCK = 32                                  # ZERO_ACT_BLOCK
ACT_NONE, ACT_GELU, ACT_SILU = 0, 1, 2          # zero_act
_ITYPES = {torch.int32: 0, torch.int64: 1}      # zero_itype

lib.zero_act_save.argtypes = [_vp, _vp, _vp, _u64, _vp, _u64, _i32, _i32, _u64, _u64, _vp]
lib.zero_act_load.argtypes = [_vp, _u64, _i32, _vp, _vp, _u64, _u64, _vp]
lib.zero_act_backward.argtypes = [_vp, _u64, _vp, _u64, _i32, _i32, _vp, _vp, _u64, _u64, _vp]
lib.zero_weight_grad.argtypes = [_vp, _i32, ctypes.c_int32, _vp, _u64, _i32, _vp, _vp, _u64, _u64,
                                 _u64, _vp, _u64, _vp]
lib.zero_weight_grad_workspace.argtypes = [_u64, _u64, _u64, ctypes.POINTER(ctypes.c_uint64)]
lib.zero_embed_lookup.argtypes = [_vp, _u64, _vp, _i32, _vp, _i32, _u64, _u64, _u64, _f32, _vp]
lib.zero_embed_grad.argtypes = [_vp, _i32, ctypes.c_int32, _vp, _u64, _i32, _vp, _i32, _u64, _u64,
                                _u64, _f32, _vp, _u64, _vp]
lib.zero_embed_grad_workspace.argtypes = [_u64, _u64, _u64, ctypes.POINTER(ctypes.c_uint64)]
_policy_args = [_vp, _vp, _vp, _vp, _u64, _vp, _u64, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _u64,
                _u64, _f32, _f32, _f32]
lib.zero_policy_loss.argtypes = [*_policy_args, _f32, _vp]
lib.zero_policy_loss_dev.argtypes = [*_policy_args, _vp, _vp]
for _f in ("zero_act_save", "zero_act_load", "zero_act_backward", "zero_weight_grad",
           "zero_weight_grad_workspace", "zero_embed_lookup", "zero_embed_grad",
           "zero_embed_grad_workspace", "zero_policy_loss", "zero_policy_loss_dev"):
    getattr(lib, _f).restype = _i32


# The checks below run on every call, so the accepted case is one expression of cheap
# tests (device index, dtype, shape, strides); what was wrong is worked out afterwards.

_get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _refuse(t, name: str, dtypes, dev, what: str) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor (got {t.device}): the kernels "
                         "read and write device memory only")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {list(dtypes)}")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    raise ValueError(f"{name} must be {what}, got shape {tuple(t.shape)} with strides "
                     f"{t.stride()}")


def _matrix(t, name: str, dtypes, shape=None, dev=None) -> tuple:
    """(pointer, row stride) of a 2-D device tensor with unit column stride, of this shape
    and on this device where they are given."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and t.dim() == 2 and
            (dev is None or t.get_device() == dev) and (shape is None or t.shape == shape)):
        _refuse(t, name, dtypes, dev, f"a matrix of shape {shape or '(rows, cols)'}")
    rows, cols = t.shape
    ld, one = t.stride()
    if one != 1 and cols > 1:
        _refuse(t, name, dtypes, dev, "a matrix with unit column stride")
    return t.data_ptr(), (ld if rows > 1 else cols)


def _flat(t, name: str, dtypes, shape, dev) -> int:
    """Pointer of a contiguous device tensor of exactly this shape."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and
            t.get_device() == dev and t.shape == shape and t.is_contiguous()):
        _refuse(t, name, dtypes, dev, f"contiguous with shape {shape}")
    return t.data_ptr()


_U8, _F32 = (torch.uint8,), (torch.float32,)


def _workspace(t, dev) -> tuple:
    if t is None:
        return None, 0
    n = t.numel() if isinstance(t, torch.Tensor) else 0
    return _flat(t, "workspace", _U8, (n,), dev), n


def _call(name: str, fn, dev: int, stream, *args) -> None:
    handle = _stream_handle(stream, torch.device("cuda", dev)) if stream is not None or \
        _raw_current_stream is None else _raw_current_stream(dev)
    if dev == _get_device():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, handle)
    if rc != 0:
        raise ZeroError(rc, name)


def _checkpoint(q, e, dev) -> tuple:
    """(q pointer, e pointer, shape) of a checkpoint."""
    if not (isinstance(q, torch.Tensor) and q.dim() == 2):
        _refuse(q, "q", _U8, dev, "a matrix of shape (rows, cols)")
    shape = q.shape
    return (_flat(q, "q", _U8, shape, dev),
            _flat(e, "e", _U8, (shape[0], -(-shape[1] // ACT_BLOCK)), dev), shape)


# ---- 8-bit activation checkpoints -------------------------------------------------

def zero_act_save(q: torch.Tensor, e: torch.Tensor, x: torch.Tensor, act: int = ACT_NONE,
                  y: torch.Tensor | None = None, stream=None) -> None:
    """Write x's checkpoint: q[rows, cols] and e[rows, ceil(cols/32)], uint8.  With an
    activation function also y = act(x); y may be x."""
    p_x, ldx = _matrix(x, "x", _FORMATS)
    dev, shape = x.get_device(), x.shape
    p_q, p_e, held = _checkpoint(q, e, dev)
    if held != shape:
        raise ValueError(f"q must have x's shape {tuple(shape)}, got {tuple(held)}")
    if act != ACT_NONE and y is None:
        raise ValueError("an activation function needs y")
    p_y, ldy = (None, 0) if y is None else _matrix(y, "y", (x.dtype,), shape, dev)
    _call("zero_act_save", lib.zero_act_save, dev, stream, p_q, p_e, p_y, ldy, p_x, ldx,
          _FORMATS[x.dtype], act, shape[0], shape[1])


def zero_act_load(x: torch.Tensor, q: torch.Tensor, e: torch.Tensor, stream=None) -> None:
    """x = the values the checkpoint (q, e) stands for."""
    p_x, ldx = _matrix(x, "x", _FORMATS)
    dev = x.get_device()
    p_q, p_e, shape = _checkpoint(q, e, dev)
    if x.shape != shape:
        raise ValueError(f"x must have q's shape {tuple(shape)}, got {tuple(x.shape)}")
    _call("zero_act_load", lib.zero_act_load, dev, stream, p_x, ldx, _FORMATS[x.dtype], p_q, p_e,
          shape[0], shape[1])


def zero_act_backward(dx: torch.Tensor, dy: torch.Tensor, q: torch.Tensor, e: torch.Tensor,
                      act: int, stream=None) -> None:
    """dx = dy * act'(v), v the checkpoint's values; dx may be dy."""
    p_dy, lddy = _matrix(dy, "dy", _FORMATS)
    dev = dy.get_device()
    p_q, p_e, shape = _checkpoint(q, e, dev)
    if dy.shape != shape:
        raise ValueError(f"dy must have q's shape {tuple(shape)}, got {tuple(dy.shape)}")
    p_dx, lddx = _matrix(dx, "dx", (dy.dtype,), shape, dev)
    _call("zero_act_backward", lib.zero_act_backward, dev, stream, p_dx, lddx, p_dy, lddy,
          _FORMATS[dy.dtype], act, p_q, p_e, shape[0], shape[1])


def _workspace_bytes(name: str, *extents) -> int:
    out = ctypes.c_uint64(0)
    rc = getattr(lib, name)(*extents, ctypes.byref(out))
    if rc != 0:
        raise ZeroError(rc, name)
    return out.value


def zero_weight_grad_workspace(tokens: int, n_out: int, n_in: int) -> int:
    """Bytes of workspace zero_weight_grad needs for these extents."""
    return _workspace_bytes("zero_weight_grad_workspace", tokens, n_out, n_in)


def zero_weight_grad(dw: torch.Tensor, dy: torch.Tensor, q: torch.Tensor, e: torch.Tensor,
                     first: bool = True, workspace: torch.Tensor | None = None,
                     stream=None) -> None:
    """dw[n_out, n_in] = (or, FP32 and not first, +=) dy^T v, v the checkpoint's values."""
    p_dy, lddy = _matrix(dy, "dy", _DTYPES)
    dev, (tokens, n_out), dt = dy.get_device(), dy.shape, dy.dtype
    p_q, p_e, (rows, n_in) = _checkpoint(q, e, dev)
    if rows != tokens:
        raise ValueError(f"q holds {rows} tokens, dy {tokens}")
    p_dw = _flat(dw, "dw", (dt, torch.float32), (n_out, n_in), dev)
    p_ws, n_ws = _workspace(workspace, dev)
    _call("zero_weight_grad", lib.zero_weight_grad, dev, stream, p_dw, _FORMATS[dw.dtype],
          int(bool(first)), p_dy, lddy, _DTYPES[dt], p_q, p_e, tokens, n_out, n_in, p_ws, n_ws)


# ---- embedding ------------------------------------------------------------------------

def zero_embed_lookup(out: torch.Tensor, table: torch.Tensor, ids: torch.Tensor,
                      scale: float = 1.0, stream=None) -> None:
    """out[t] = scale * table[ids[t]]; zeros where ids[t] is outside the table."""
    p_out, ldo = _matrix(out, "out", _FORMATS)
    dev, (tokens, width), dt = out.get_device(), out.shape, out.dtype
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be a 2-D tensor (vocab, width)")
    vocab = table.shape[0]
    p_t = _flat(table, "table", (dt,), (vocab, width), dev)
    p_i = _flat(ids, "ids", _ITYPES, (tokens,), dev)
    _call("zero_embed_lookup", lib.zero_embed_lookup, dev, stream, p_out, ldo, p_t, _FORMATS[dt],
          p_i, _ITYPES[ids.dtype], tokens, vocab, width, scale)


def zero_embed_grad_workspace(tokens: int, vocab: int, width: int) -> int:
    """Bytes of workspace zero_embed_grad needs for these extents."""
    return _workspace_bytes("zero_embed_grad_workspace", tokens, vocab, width)


def zero_embed_grad(dw: torch.Tensor, dy: torch.Tensor, ids: torch.Tensor, scale: float = 1.0,
                    first: bool = True, workspace: torch.Tensor | None = None,
                    stream=None) -> None:
    """dw[v] = scale * sum of dy[t] over ids[t] == v; FP32 and not first: added to dw's rows."""
    p_dy, lddy = _matrix(dy, "dy", _DTYPES)
    dev, (tokens, width), dt = dy.get_device(), dy.shape, dy.dtype
    if not isinstance(dw, torch.Tensor) or dw.dim() != 2:
        raise ValueError("dw must be a 2-D tensor (vocab, width)")
    vocab = dw.shape[0]
    p_dw = _flat(dw, "dw", (dt, torch.float32), (vocab, width), dev)
    p_i = _flat(ids, "ids", _ITYPES, (tokens,), dev)
    p_ws, n_ws = _workspace(workspace, dev)
    _call("zero_embed_grad", lib.zero_embed_grad, dev, stream, p_dw, _FORMATS[dw.dtype],
          int(bool(first)), p_dy, lddy, _DTYPES[dt], p_i, _ITYPES[ids.dtype], tokens, vocab, width,
          scale, p_ws, n_ws)


# ---- policy loss ------------------------------------------------------------------------

def _policy(loss, token_loss, logp, logits, targets, advantage, weight, old_logp, ref_logp,
            dlogits, clip_low, clip_high, kl_coef):
    p_z, ld = _matrix(logits, "logits", _FORMATS)
    dev, shape, dt = logits.get_device(), logits.shape, logits.dtype
    one, rows = (1,), shape[:1]
    p_d, ldd = (None, 0) if dlogits is None else \
        _matrix(dlogits, "dlogits", (dt,), shape, dev)
    return dev, (_flat(loss, "loss", _F32, one, dev),
                 _flat(token_loss, "token_loss", _F32, rows, dev),
                 _flat(logp, "logp", _F32, rows, dev), p_d, ldd, p_z, ld, _FORMATS[dt],
                 _flat(targets, "targets", _ITYPES, rows, dev), _ITYPES[targets.dtype],
                 None if old_logp is None else _flat(old_logp, "old_logp", _F32, rows, dev),
                 None if ref_logp is None else _flat(ref_logp, "ref_logp", _F32, rows, dev),
                 _flat(advantage, "advantage", _F32, rows, dev),
                 _flat(weight, "weight", _F32, rows, dev), shape[0], shape[1], clip_low,
                 clip_high, kl_coef)


def zero_policy_loss(loss: torch.Tensor, token_loss: torch.Tensor, logp: torch.Tensor,
                     logits: torch.Tensor, targets: torch.Tensor, advantage: torch.Tensor,
                     weight: torch.Tensor, *, old_logp: torch.Tensor | None = None,
                     ref_logp: torch.Tensor | None = None, clip_low: float, clip_high: float,
                     kl_coef: float, loss_scale: float, dlogits: torch.Tensor | None = None,
                     stream=None) -> None:
    """Clipped policy loss with a KL term over sampled tokens and, with dlogits, its gradient
    times loss_scale; dlogits may be logits."""
    dev, args = _policy(loss, token_loss, logp, logits, targets, advantage, weight, old_logp,
                        ref_logp, dlogits, clip_low, clip_high, kl_coef)
    _call("zero_policy_loss", lib.zero_policy_loss, dev, stream, *args, loss_scale)


def zero_policy_loss_dev(loss: torch.Tensor, token_loss: torch.Tensor, logp: torch.Tensor,
                         logits: torch.Tensor, targets: torch.Tensor, advantage: torch.Tensor,
                         weight: torch.Tensor, *, old_logp: torch.Tensor | None = None,
                         ref_logp: torch.Tensor | None = None, clip_low: float,
                         clip_high: float, kl_coef: float, ctl: torch.Tensor,
                         dlogits: torch.Tensor | None = None, stream=None) -> None:
    """zero_policy_loss with the loss scale read from the device control block."""
    dev, args = _policy(loss, token_loss, logp, logits, targets, advantage, weight, old_logp,
                        ref_logp, dlogits, clip_low, clip_high, kl_coef)
    _call("zero_policy_loss_dev", lib.zero_policy_loss_dev, dev, stream, *args,
          _ctl_ptr(ctl, logits.device))
