"""Binding of the training operators: layer norm, dropout with its residual,
cross entropy of a linear head.

The functions pass their arguments on to the CPython module built from
``csrc/zr_torch.cpp``, which reads the tensors, allocates outputs and
workspace, and calls the C entry points of ``include/zr.h`` on the current
stream.  There is no CPU fallback: if the module is missing or a tensor is not
on a CUDA device, calls raise.
"""
from __future__ import annotations

import importlib.machinery
import importlib.util
import os

import torch  # noqa: F401  (the module links against it)

import broadcast_elementwise_shape_gb300 as _zr

from .build import TORCH_LIB as _PATH

_module = None


def _c():
    """The loaded binding module; raises if it has not been built."""
    global _module
    if _module is None:
        if not os.path.exists(_PATH):
            raise RuntimeError(f"zr binding not built ({_PATH}); run "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        loader = importlib.machinery.ExtensionFileLoader("zr_torch", _PATH)
        spec = importlib.util.spec_from_file_location("zr_torch", _PATH, loader=loader)
        module = importlib.util.module_from_spec(spec)
        loader.exec_module(module)
        _module = module
    return _module


def _out(result, where):
    """The call's tensors; an int is the status of a call that failed."""
    if type(result) is int:
        raise _zr.ZrError(result, where)
    return result


def zr_layer_norm_fwd(x, gamma=None, beta=None, eps=1e-5, out=None, keep_stats=True):
    """(y, mean, rstd) of layer norm over x's last dim: y = (x - mean) * rstd *
    gamma + beta.  mean and rstd are float32 of the leading shape, or None with
    ``keep_stats`` false.  ``out`` may be a preallocated (strided) tensor of
    x's shape, or x itself."""
    return _out(_c().layer_norm_fwd(x, gamma, beta, eps, out, bool(keep_stats)), "zr_layer_norm_fwd")


def zr_layer_norm_bwd(grad_out, x, gamma, mean, rstd, want=(True, True, True),
                      grads=(None, None, None), workspace=None):
    """(grad_x, grad_gamma, grad_beta) of layer norm given grad_out and the
    forward's mean and rstd.  ``gamma`` may be None (1); ``grads`` may hold
    preallocated outputs (grad_x of any strides, or grad_out or x itself)."""
    wx, wg, wb = want
    return _out(_c().layer_norm_bwd(grad_out, x, gamma, mean, rstd, bool(wx), bool(wg), bool(wb), *grads,
                                    workspace), "zr_layer_norm_bwd")


def zr_dropout_fwd(x, p, seed, offset=0, residual=None, out=None, device_offset=None):
    """out = residual + (keep ? x / (1 - p) : 0).  The mask is a function of
    (seed, offset, row-major element index) alone: a call uses the counters
    offset .. offset + ceil(numel / 4) - 1.  ``device_offset`` (one int64 on
    the device) is added to ``offset`` when the kernel runs.  ``out`` may be a
    preallocated (strided) tensor, x, or the residual."""
    return _out(_c().dropout_fwd(x, p, seed, offset, residual, out, device_offset), "zr_dropout_fwd")


def zr_dropout_bwd(grad_out, p, seed, offset=0, grad_x=None, device_offset=None):
    """grad_x = keep ? grad_out / (1 - p) : 0 with the forward's mask."""
    return _out(_c().dropout_bwd(grad_out, p, seed, offset, grad_x, device_offset), "zr_dropout_bwd")


_REDUCTION = {"none": 0, "mean": 1, "sum": 2}  # zr_reduction


def _reduction(reduction):
    red = _REDUCTION.get(reduction)
    if red is None:
        raise ValueError(f"reduction must be one of {sorted(_REDUCTION)}")
    return red


def zr_linear_xent_fwd(x, w, labels, reduction="mean", ignore_index=-100, workspace=None):
    """(loss, lse) of the softmax cross entropy of logits x w^T, which are
    never stored: x [..., D], w [V, D], labels x's leading shape.  loss is a
    float32 scalar, or per row with reduction "none"; lse (float32 per row) is
    what the backward takes."""
    return _out(_c().linear_xent_fwd(x, w, labels, _reduction(reduction), ignore_index, workspace),
                "zr_linear_xent_fwd")


def zr_linear_xent_bwd(grad_loss, x, w, labels, lse, reduction="mean", ignore_index=-100,
                       want=(True, True), grads=(None, None), workspace=None):
    """(grad_x, grad_w) of zr_linear_xent_fwd's loss given grad_loss (float32,
    one element, or one per row with reduction "none", views too) and the
    forward's lse.
    ``grads`` may hold preallocated contiguous outputs."""
    wx, ww = want
    return _out(_c().linear_xent_bwd(grad_loss, x, w, labels, lse, _reduction(reduction), ignore_index,
                                     bool(wx), bool(ww), *grads, workspace), "zr_linear_xent_bwd")
