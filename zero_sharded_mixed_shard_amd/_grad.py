"""ctypes binding of the gradient operators (see include/zero_shard_grad.h for the contract)."""
from __future__ import annotations

import ctypes

import torch

from ._binding import (_DTYPES, _FORMATS, _ctl_ptr, _f32, _i32, _stream_handle, _u64, _vp,
                       ZeroError, lib)

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


def _on_device(t, name: str, dtypes, device) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor (got {t.device}): the kernels "
                         "read and write device memory only")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {list(dtypes)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _matrix(t, name: str, dtypes, shape=None, device=None) -> tuple:
    """(pointer, row stride) of a 2-D device tensor with unit column stride."""
    _on_device(t, name, dtypes, device)
    if t.dim() != 2 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{name} must have shape {tuple(shape) if shape else '(rows, cols)'}, "
                         f"got {tuple(t.shape)}")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride")
    return t.data_ptr(), (t.stride(0) if rows > 1 else cols)


def _flat(t, name: str, dtypes, shape, device) -> int:
    """Pointer of a contiguous device tensor of exactly this shape."""
    _on_device(t, name, dtypes, device)
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {tuple(shape)}, got "
                         f"{tuple(t.shape)} with strides {t.stride()}")
    return t.data_ptr()


def _workspace(t, device) -> tuple:
    if t is None:
        return None, 0
    _on_device(t, "workspace", (torch.uint8,), device)
    if t.dim() != 1 or not t.is_contiguous():
        raise ValueError("workspace must be a 1-D contiguous uint8 tensor")
    return t.data_ptr(), t.numel()


def _call(name: str, device, stream, *args) -> None:
    fn = getattr(lib, name)
    if device.index == torch.cuda.current_device():
        rc = fn(*args, _stream_handle(stream, device))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, _stream_handle(stream, device))
    if rc != 0:
        raise ZeroError(rc, name)


def _checkpoint(q, e, device) -> tuple:
    """(q pointer, e pointer, rows, cols) of a checkpoint."""
    _on_device(q, "q", (torch.uint8,), device)
    if q.dim() != 2:
        raise ValueError(f"q must have shape (rows, cols), got {tuple(q.shape)}")
    rows, cols = q.shape
    p_q = _flat(q, "q", (torch.uint8,), (rows, cols), device)
    p_e = _flat(e, "e", (torch.uint8,), (rows, -(-cols // ACT_BLOCK)), device)
    return p_q, p_e, rows, cols


# ---- 8-bit activation checkpoints -------------------------------------------------

def zero_act_save(q: torch.Tensor, e: torch.Tensor, x: torch.Tensor, act: int = ACT_NONE,
                  y: torch.Tensor | None = None, stream=None) -> None:
    """Write x's checkpoint: q[rows, cols] and e[rows, ceil(cols/32)], uint8.  With an
    activation function also y = act(x); y may be x."""
    p_x, ldx = _matrix(x, "x", _FORMATS)
    dev, (rows, cols) = x.device, x.shape
    p_q, p_e, *shape = _checkpoint(q, e, dev)
    if shape != [rows, cols]:
        raise ValueError(f"q must have x's shape {(rows, cols)}, got {tuple(shape)}")
    p_y, ldy = (None, 0) if y is None else _matrix(y, "y", (x.dtype,), x.shape, dev)
    if act != ACT_NONE and y is None:
        raise ValueError("an activation function needs y")
    _call("zero_act_save", dev, stream, p_q, p_e, p_y, ldy, p_x, ldx, _FORMATS[x.dtype], act,
          rows, cols)


def zero_act_load(x: torch.Tensor, q: torch.Tensor, e: torch.Tensor, stream=None) -> None:
    """x = the values the checkpoint (q, e) stands for."""
    p_x, ldx = _matrix(x, "x", _FORMATS)
    p_q, p_e, rows, cols = _checkpoint(q, e, x.device)
    if tuple(x.shape) != (rows, cols):
        raise ValueError(f"x must have q's shape {(rows, cols)}, got {tuple(x.shape)}")
    _call("zero_act_load", x.device, stream, p_x, ldx, _FORMATS[x.dtype], p_q, p_e, rows, cols)


def zero_act_backward(dx: torch.Tensor, dy: torch.Tensor, q: torch.Tensor, e: torch.Tensor,
                      act: int, stream=None) -> None:
    """dx = dy * act'(v), v the checkpoint's values; dx may be dy."""
    p_dy, lddy = _matrix(dy, "dy", _FORMATS)
    dev = dy.device
    p_q, p_e, rows, cols = _checkpoint(q, e, dev)
    if tuple(dy.shape) != (rows, cols):
        raise ValueError(f"dy must have q's shape {(rows, cols)}, got {tuple(dy.shape)}")
    p_dx, lddx = _matrix(dx, "dx", (dy.dtype,), dy.shape, dev)
    _call("zero_act_backward", dev, stream, p_dx, lddx, p_dy, lddy, _FORMATS[dy.dtype], act, p_q,
          p_e, rows, cols)


def _workspace_bytes(name: str, *extents) -> int:
    out = ctypes.c_uint64(0)
    rc = getattr(lib, name)(*extents, ctypes.byref(out))
    if rc != 0:
        raise ZeroError(rc, name)
    return out.value


def zero_weight_grad_workspace(tokens: int, n_out: int, n_in: int) -> int:
    """Bytes of workspace zero_weight_grad needs for these extents."""
    return _workspace_bytes("zero_weight_grad_workspace", tokens, n_out, n_in)


def _target_dtypes(dtype) -> tuple:
    return (dtype, torch.float32)


def zero_weight_grad(dw: torch.Tensor, dy: torch.Tensor, q: torch.Tensor, e: torch.Tensor,
                     first: bool = True, workspace: torch.Tensor | None = None,
                     stream=None) -> None:
    """dw[n_out, n_in] = (or, FP32 and not first, +=) dy^T v, v the checkpoint's values."""
    p_dy, lddy = _matrix(dy, "dy", _DTYPES)
    dev, (tokens, n_out) = dy.device, dy.shape
    p_q, p_e, rows, n_in = _checkpoint(q, e, dev)
    if rows != tokens:
        raise ValueError(f"q holds {rows} tokens, dy {tokens}")
    p_dw = _flat(dw, "dw", _target_dtypes(dy.dtype), (n_out, n_in), dev)
    p_ws, n_ws = _workspace(workspace, dev)
    _call("zero_weight_grad", dev, stream, p_dw, _FORMATS[dw.dtype], int(bool(first)), p_dy, lddy,
          _DTYPES[dy.dtype], p_q, p_e, tokens, n_out, n_in, p_ws, n_ws)


# ---- embedding ------------------------------------------------------------------------

def zero_embed_lookup(out: torch.Tensor, table: torch.Tensor, ids: torch.Tensor,
                      scale: float = 1.0, stream=None) -> None:
    """out[t] = scale * table[ids[t]]; zeros where ids[t] is outside the table."""
    p_out, ldo = _matrix(out, "out", _FORMATS)
    dev, (tokens, width) = out.device, out.shape
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be a 2-D tensor (vocab, width)")
    vocab = table.shape[0]
    p_t = _flat(table, "table", (out.dtype,), (vocab, width), dev)
    p_i = _flat(ids, "ids", _ITYPES, (tokens,), dev)
    _call("zero_embed_lookup", dev, stream, p_out, ldo, p_t, _FORMATS[out.dtype], p_i,
          _ITYPES[ids.dtype], tokens, vocab, width, scale)


def zero_embed_grad_workspace(tokens: int, vocab: int, width: int) -> int:
    """Bytes of workspace zero_embed_grad needs for these extents."""
    return _workspace_bytes("zero_embed_grad_workspace", tokens, vocab, width)


def zero_embed_grad(dw: torch.Tensor, dy: torch.Tensor, ids: torch.Tensor, scale: float = 1.0,
                    first: bool = True, workspace: torch.Tensor | None = None,
                    stream=None) -> None:
    """dw[v] = scale * sum of dy[t] over ids[t] == v; FP32 and not first: added to dw's rows."""
    p_dy, lddy = _matrix(dy, "dy", _DTYPES)
    dev, (tokens, width) = dy.device, dy.shape
    if not isinstance(dw, torch.Tensor) or dw.dim() != 2:
        raise ValueError("dw must be a 2-D tensor (vocab, width)")
    vocab = dw.shape[0]
    p_dw = _flat(dw, "dw", _target_dtypes(dy.dtype), (vocab, width), dev)
    p_i = _flat(ids, "ids", _ITYPES, (tokens,), dev)
    p_ws, n_ws = _workspace(workspace, dev)
    _call("zero_embed_grad", dev, stream, p_dw, _FORMATS[dw.dtype], int(bool(first)), p_dy, lddy,
          _DTYPES[dy.dtype], p_i, _ITYPES[ids.dtype], tokens, vocab, width, scale, p_ws, n_ws)


# ---- policy loss ------------------------------------------------------------------------

def _policy(loss, token_loss, logp, logits, targets, advantage, weight, old_logp, ref_logp,
            dlogits, clip_low, clip_high, kl_coef):
    p_z, ld = _matrix(logits, "logits", _FORMATS)
    dev, (rows, vocab) = logits.device, logits.shape
    f32 = (torch.float32,)

    def rows_of(t, name):
        return None if t is None else _flat(t, name, f32, (rows,), dev)

    p_d, ldd = (None, 0) if dlogits is None else \
        _matrix(dlogits, "dlogits", (logits.dtype,), logits.shape, dev)
    for t, name in ((token_loss, "token_loss"), (logp, "logp"), (advantage, "advantage"),
                    (weight, "weight")):
        _on_device(t, name, f32, dev)
    return dev, (_flat(loss, "loss", f32, (1,), dev), rows_of(token_loss, "token_loss"),
                 rows_of(logp, "logp"), p_d, ldd, p_z, ld, _FORMATS[logits.dtype],
                 _flat(targets, "targets", _ITYPES, (rows,), dev), _ITYPES[targets.dtype],
                 rows_of(old_logp, "old_logp"), rows_of(ref_logp, "ref_logp"),
                 rows_of(advantage, "advantage"), rows_of(weight, "weight"), rows, vocab,
                 clip_low, clip_high, kl_coef)


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
    _call("zero_policy_loss", dev, stream, *args, loss_scale)


def zero_policy_loss_dev(loss: torch.Tensor, token_loss: torch.Tensor, logp: torch.Tensor,
                         logits: torch.Tensor, targets: torch.Tensor, advantage: torch.Tensor,
                         weight: torch.Tensor, *, old_logp: torch.Tensor | None = None,
                         ref_logp: torch.Tensor | None = None, clip_low: float,
                         clip_high: float, kl_coef: float, ctl: torch.Tensor,
                         dlogits: torch.Tensor | None = None, stream=None) -> None:
    """zero_policy_loss with the loss scale read from the device control block."""
    dev, args = _policy(loss, token_loss, logp, logits, targets, advantage, weight, old_logp,
                        ref_logp, dlogits, clip_low, clip_high, kl_coef)
    _call("zero_policy_loss_dev", dev, stream, *args, _ctl_ptr(ctl, dev))
