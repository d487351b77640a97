"""The group norm with an activation, channels last -- Python binding of the entry points
that ``include/wkv7.h`` documents as ``wkv7_gnorm_*``.

Contiguous float32 or bfloat16 device tensors [..., D]; gamma and beta are float32 [D].
The work is enqueued on the device's current torch stream.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

from . import GnormDesc, _dtype_code, _ptr, _torch, lib
from .mixers import _call, _maybe, _result, _same, _scratch


class GnormGrads(NamedTuple):
    """Gradients of ``gnorm_backward``; dgamma, dbeta, dz are None without theirs."""
    dx: object
    dgamma: object
    dbeta: object
    dz: object


def _inputs(x, groups: int, gamma, beta, z, gate_first: bool, silu: bool, center: bool, eps: float):
    torch = _torch()
    code = _dtype_code(x)
    if x.dim() < 1:
        raise ValueError("x is [..., D]")
    D = x.shape[-1]
    rows = x.numel() // D if D else 0
    _same(x, "x", x.shape, x.dtype, x.device)
    _maybe(z, "z", x.shape, x.dtype, x.device)
    _maybe(gamma, "gamma", (D,), torch.float32, x.device)
    _maybe(beta, "beta", (D,), torch.float32, x.device)
    if gate_first and z is None:
        raise ValueError("gate_first goes with z")
    return GnormDesc(rows, D, groups, code, 1 if center else 0, 1 if silu else 0,
                     0 if z is None else 2 if gate_first else 1, eps)


def gnorm_forward(x, groups: int, gamma=None, beta=None, *, z=None, gate_first: bool = False, silu: bool = False,
                  center: bool = True, eps: float = 1e-5, out=None):
    """Per row of ``x`` [..., D], over each of ``groups`` groups of neighbouring channels
    (wkv7_gnorm_forward): u = x, or x z sigmoid(z) with ``z`` and ``gate_first``; n = (u -
    mean) / sqrt(var + eps), or u / sqrt(mean u^2 + eps) with ``center=False``; o = gamma n +
    beta; y = o, or o sigmoid(o) with ``silu``; then times z sigmoid(z) with ``z`` and not
    ``gate_first``.  Returns y.  ``groups`` = heads is the norm of a read-out."""
    d = _inputs(x, groups, gamma, beta, z, gate_first, silu, center, eps)
    y = _result(out, "out", x, (x, z, gamma, beta))
    _call("wkv7_gnorm_forward", x.device, ctypes.byref(d), _ptr(gamma), _ptr(beta), _ptr(x), _ptr(z), _ptr(y))
    return y


def gnorm_backward(x, dy, groups: int, gamma=None, beta=None, *, z=None, gate_first: bool = False,
                   silu: bool = False, center: bool = True, eps: float = 1e-5, workspace=None) -> GnormGrads:
    """Gradients of ``<dy, y>`` (wkv7_gnorm_backward)."""
    torch = _torch()
    d = _inputs(x, groups, gamma, beta, z, gate_first, silu, center, eps)
    _same(dy, "dy", x.shape, x.dtype, x.device)
    like = lambda p: None if p is None else torch.empty_like(p)   # noqa: E731
    grads = GnormGrads(torch.empty_like(x), like(gamma), like(beta), like(z))
    ws, wsb, _held = _scratch(workspace, lib().wkv7_gnorm_backward_workspace_bytes(ctypes.byref(d)), x.device)
    _call("wkv7_gnorm_backward", x.device, ctypes.byref(d), _ptr(gamma), _ptr(beta), _ptr(x), _ptr(z), _ptr(dy),
          _ptr(grads.dx), _ptr(grads.dz), _ptr(grads.dgamma), _ptr(grads.dbeta), ws, wsb)
    return grads
