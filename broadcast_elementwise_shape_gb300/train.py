"""Binding of the training operators: layer norm, dropout with its residual,
cross entropy of a linear head.

Their calls are short, so what the binding costs counts: a call hands over
its arguments as one packed array (``include/zr_packed.h``) instead of a
dozen ctypes objects (on a Grace core, layer norm of one row took 41 us per
call that way and 4 us of it in the C function).
"""
from __future__ import annotations

import ctypes
import struct

import torch

import broadcast_elementwise_shape_gb300 as _zr

_F32, _BF16 = torch.float32, torch.bfloat16
_CODE = {_F32: 0, _BF16: 1}  # zr_dtype
_NONE = (0, 0)               # a tensor that is not given
_ERR_WORKSPACE = -7
_raw_stream = torch._C._cuda_getCurrentRawStream
_empty = torch.empty


def _words(t):
    """A tensor's words: data address, ndim, sizes, strides."""
    shape = t.shape
    return (t.data_ptr(), len(shape), *shape, *t.stride())


def _code(t, *others):
    """The zr_dtype that all given tensors share, on one CUDA device."""
    dt = t.dtype
    code = _CODE.get(dt)
    if code is None:
        raise TypeError(f"zr operands must be float32 or bfloat16 (got {dt})")
    for o in others:
        if o is not None and o.dtype != dt:
            raise TypeError(f"operands mix element types {dt} and {o.dtype}")
    for o in (t, *others):
        if o is not None and not o.is_cuda:
            raise ValueError("zr operands must be CUDA tensors")
    return code


def _same_shape(t, shape, what):
    if t.shape != shape:
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _stats(t, shape, what):
    """A float32 tensor that must be dense over `shape`."""
    if t.dtype != _F32:
        raise TypeError(f"{what} must be float32")
    if not t.is_cuda:
        raise ValueError("zr operands must be CUDA tensors")
    _same_shape(t, shape, what)
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _fail(rc, where):
    raise _zr.ZrError(rc, where)


def _pack(scalar, words):
    return struct.pack(f"d{len(words)}q", scalar, *words)


_TRY = 1 << 16  # bytes: enough for short calls, which then take one call instead of two


def _with_workspace(fn, name, words, at, workspace, device):
    """Call with the caller's workspace or a small one; where that is too
    little, once more with what the call asked for.  words[at] and
    words[at + 1] are the workspace's address and size."""
    if workspace is None or workspace.numel() < 16:
        workspace = _empty(_TRY, dtype=torch.uint8, device=device)
    n = workspace.numel()
    words[at] = workspace.data_ptr()
    words[at + 1] = n
    need = ctypes.c_int64(0)
    rc = fn(_pack(0.0, words), ctypes.byref(need))
    if rc == _ERR_WORKSPACE and need.value > n:
        workspace = _empty(need.value, dtype=torch.uint8, device=device)
        words[at] = workspace.data_ptr()
        words[at + 1] = need.value
        rc = fn(_pack(0.0, words), ctypes.byref(need))
    if rc:
        _fail(rc, name)


def zr_layer_norm_fwd(x, gamma=None, beta=None, eps=1e-5, out=None, keep_stats=True):
    """(y, mean, rstd) of layer norm over x's last dim: y = (x - mean) * rstd *
    gamma + beta.  mean and rstd are float32 of the leading shape, or None with
    ``keep_stats`` false.  ``out`` may be a preallocated (strided) tensor of
    x's shape, or x itself."""
    shape = x.shape
    dev = x.device
    if out is None:
        code = _code(x, gamma, beta)
        out = _empty(shape, dtype=x.dtype, device=dev)
    else:
        code = _code(x, gamma, beta, out)
        _same_shape(out, shape, "out")
    mean = rstd = None
    if keep_stats:
        lead = shape[:-1]
        mean = _empty(lead, dtype=_F32, device=dev)
        rstd = _empty(lead, dtype=_F32, device=dev)
    words = (code, _raw_stream(dev.index), mean.data_ptr() if keep_stats else 0,
             rstd.data_ptr() if keep_stats else 0, *_words(x),
             *(_NONE if gamma is None else _words(gamma)),
             *(_NONE if beta is None else _words(beta)), *_words(out))
    rc = _zr.lib().zr_packed_layer_norm_fwd(_pack(eps, words))
    if rc:
        _fail(rc, "zr_layer_norm_fwd")
    return out, mean, rstd


def zr_layer_norm_bwd(grad_out, x, gamma, mean, rstd, want=(True, True, True),
                      grads=(None, None, None), workspace=None):
    """(grad_x, grad_gamma, grad_beta) of layer norm given grad_out and the
    forward's mean and rstd.  ``gamma`` may be None (1); ``grads`` may hold
    preallocated outputs (grad_x of any strides, or grad_out or x itself)."""
    shape, dev, dt = x.shape, x.device, x.dtype
    gx, gg, gb = grads
    code = _code(x, grad_out, gamma, gx, gg, gb)
    lead, width = shape[:-1], shape[-1:]
    pm, pr = _stats(mean, lead, "mean"), _stats(rstd, lead, "rstd")
    if gx is None:
        gx = _empty(shape, dtype=dt, device=dev) if want[0] else None
    else:
        _same_shape(gx, shape, "grad_x")
    if gg is None:
        gg = _empty(width, dtype=dt, device=dev) if want[1] else None
    else:
        _dense(gg, width, "grad_gamma")
    if gb is None:
        gb = _empty(width, dtype=dt, device=dev) if want[2] else None
    else:
        _dense(gb, width, "grad_beta")
    words = [code, _raw_stream(dev.index), pm, pr, 0 if gg is None else gg.data_ptr(),
             0 if gb is None else gb.data_ptr(), 0, 0, *_words(grad_out), *_words(x),
             *(_NONE if gamma is None else _words(gamma)), *(_NONE if gx is None else _words(gx))]
    _with_workspace(_zr.lib().zr_packed_layer_norm_bwd, "zr_layer_norm_bwd", words, 6, workspace, dev)
    return gx, gg, gb


def _dense(t, shape, what):
    _same_shape(t, shape, what)
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")


def _word64(v):
    """An unsigned 64-bit value (taken modulo 2^64) as a signed word."""
    v = int(v) & 0xFFFFFFFFFFFFFFFF
    return v - (1 << 64) if v >> 63 else v


def _device_offset(t):
    if t is None:
        return 0
    if t.dtype != torch.int64 or t.numel() != 1:
        raise TypeError("device_offset must be one int64 element")
    if not t.is_cuda:
        raise ValueError("zr operands must be CUDA tensors")
    return t.data_ptr()


def zr_dropout_fwd(x, p, seed, offset=0, residual=None, out=None, device_offset=None):
    """out = residual + (keep ? x / (1 - p) : 0).  The mask is a function of
    (seed, offset, row-major element index) alone: a call uses the counters
    offset .. offset + ceil(numel / 4) - 1.  ``device_offset`` (one int64 on
    the device) is added to ``offset`` when the kernel runs.  ``out`` may be a
    preallocated (strided) tensor, x, or the residual."""
    at = _device_offset(device_offset)
    if residual is not None:
        _same_shape(residual, x.shape, "residual")
    if out is not None:
        _same_shape(out, x.shape, "out")
    code = _code(x, residual, out)
    dev = x.device
    if out is None:
        out = _empty(x.shape, dtype=x.dtype, device=dev)
    words = (code, _raw_stream(dev.index), _word64(seed), _word64(offset), at, *_words(x),
             *(_NONE if residual is None else _words(residual)), *_words(out))
    rc = _zr.lib().zr_packed_dropout_fwd(_pack(p, words))
    if rc:
        _fail(rc, "zr_dropout_fwd")
    return out


def zr_dropout_bwd(grad_out, p, seed, offset=0, grad_x=None, device_offset=None):
    """grad_x = keep ? grad_out / (1 - p) : 0 with the forward's mask."""
    at = _device_offset(device_offset)
    if grad_x is not None:
        _same_shape(grad_x, grad_out.shape, "grad_x")
    code = _code(grad_out, grad_x)
    dev = grad_out.device
    if grad_x is None:
        grad_x = _empty(grad_out.shape, dtype=grad_out.dtype, device=dev)
    words = (code, _raw_stream(dev.index), _word64(seed), _word64(offset), at, *_words(grad_out),
             *_words(grad_x))
    rc = _zr.lib().zr_packed_dropout_bwd(_pack(p, words))
    if rc:
        _fail(rc, "zr_dropout_bwd")
    return grad_x


_REDUCTION = {"none": 0, "mean": 1, "sum": 2}


def _reduction(reduction):
    red = _REDUCTION.get(reduction)
    if red is None:
        raise ValueError(f"reduction must be one of {sorted(_REDUCTION)}")
    return red


def _label_type(labels, lead):
    if labels.dtype not in (torch.int64, torch.int32):
        raise TypeError("labels must be int32 or int64")
    if not labels.is_cuda:
        raise ValueError("zr operands must be CUDA tensors")
    _same_shape(labels, lead, "labels")
    return 1 if labels.dtype == torch.int64 else 0


def zr_linear_xent_fwd(x, w, labels, reduction="mean", ignore_index=-100, workspace=None):
    """(loss, lse) of the softmax cross entropy of logits x w^T, which are
    never stored: x [..., D], w [V, D], labels x's leading shape.  loss is a
    float32 scalar, or per row with reduction "none"; lse (float32 per row) is
    what the backward takes."""
    red = _reduction(reduction)
    code = _code(x, w)
    lead, dev = x.shape[:-1], x.device
    it = _label_type(labels, lead)
    loss = _empty(() if red else lead, dtype=_F32, device=dev)
    lse = _empty(lead, dtype=_F32, device=dev)
    words = [code, _raw_stream(dev.index), it, int(ignore_index), red, loss.data_ptr(),
             lse.data_ptr(), 0, 0, *_words(x), *_words(w), *_words(labels)]
    _with_workspace(_zr.lib().zr_packed_linear_xent_fwd, "zr_linear_xent_fwd", words, 7, workspace, dev)
    return loss, lse


def zr_linear_xent_bwd(grad_loss, x, w, labels, lse, reduction="mean", ignore_index=-100,
                       want=(True, True), grads=(None, None), workspace=None):
    """(grad_x, grad_w) of zr_linear_xent_fwd's loss given grad_loss (float32,
    one element, or one per row with reduction "none") and the forward's lse.
    ``grads`` may hold preallocated contiguous outputs."""
    red = _reduction(reduction)
    gx, gw = grads
    code = _code(x, w, gx, gw)
    lead, dev = x.shape[:-1], x.device
    it = _label_type(labels, lead)
    pl = _stats(lse, lead, "lse")
    pg = _stats(grad_loss, grad_loss.shape, "grad_loss")
    if grad_loss.numel() != (1 if red else lse.numel()):
        raise ValueError(f"grad_loss has {grad_loss.numel()} elements, expected "
                         f"{1 if red else lse.numel()}")
    if gx is None:
        gx = _empty(x.shape, dtype=x.dtype, device=dev) if want[0] else None
    else:
        _dense(gx, x.shape, "grad_x")
    if gw is None:
        gw = _empty(w.shape, dtype=w.dtype, device=dev) if want[1] else None
    else:
        _dense(gw, w.shape, "grad_w")
    words = [code, _raw_stream(dev.index), it, int(ignore_index), red, pg, pl,
             0 if gx is None else gx.data_ptr(), 0 if gw is None else gw.data_ptr(), 0, 0,
             *_words(x), *_words(w), *_words(labels)]
    _with_workspace(_zr.lib().zr_packed_linear_xent_bwd, "zr_linear_xent_bwd", words, 9, workspace, dev)
    return gx, gw
