"""The short causal convolution and the selective state-space scan -- Python binding.

Argument checks and marshalling for the entry points that ``include/wkv7.h``
documents under the same names.  Token tensors are contiguous float32 or
bfloat16 device tensors, [B, T, D] (one token: [B, D]); states and learned
vectors are float32.  All tensors of a call lie on one device; the work is
enqueued on that device's current torch stream.  ``lengths`` (int32 [B]) gives
the valid tokens of every row of a padded batch: inputs behind a row's length
are not used, outputs there are zero, states are those after its last token.
Outputs may not share memory with inputs.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

from . import (WKV7_OK, ConvDesc, SsmDesc, SsmGradPointers, SsmParams, WKV7Error, _dtype_code, _ptr,
               _torch, lib)


def _same(t, name: str, shape, dtype, device):
    """t, checked to be a contiguous device tensor of this shape and type on `device`."""
    if t.device != device or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous device tensor on {device}")
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name}: {tuple(t.shape)} {t.dtype} instead of {tuple(shape)} {dtype}")
    return t


def _maybe(t, name: str, shape, dtype, device):
    return t if t is None else _same(t, name, shape, dtype, device)


def _result(out, name: str, like, inputs):
    """A new tensor like `like`, or the caller's `out` if it overlaps none of the inputs."""
    if out is None:
        return _torch().empty_like(like)
    _same(out, name, like.shape, like.dtype, like.device)
    lo, hi = out.data_ptr(), out.data_ptr() + out.numel() * out.element_size()
    for t in inputs:
        if t is not None and t.data_ptr() < hi and lo < t.data_ptr() + t.numel() * t.element_size():
            raise ValueError(f"{name} overlaps an input")
    return out


def _scratch(workspace, need: int, device):
    """(pointer, bytes) of the caller's workspace or of a new one."""
    torch = _torch()
    if workspace is None:
        workspace = torch.empty((need + 15) // 16 * 16, device=device, dtype=torch.uint8) if need else None
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous device tensor on {device}")
    if workspace is None:
        return None, 0, None
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _call(name: str, device, *args):
    """The entry point on `device`'s current stream."""
    torch = _torch()
    # The raw handle: making a Stream object of it takes 2 us, a fifth of a single token's call.
    stream = torch._C._cuda_getCurrentRawStream(device.index)
    if device.index == torch.cuda.current_device():
        st = getattr(lib(), name)(*args, stream)
    else:
        with torch.cuda.device(device):
            st = getattr(lib(), name)(*args, stream)
    if st != WKV7_OK:
        raise WKV7Error(st, name)


def _tokens(x, dims: int):
    if x.dim() != dims:
        raise ValueError(f"x must have {dims} dimensions, not {x.dim()}")
    code = _dtype_code(x)
    _same(x, "x", x.shape, x.dtype, x.device)
    return code


# ---- the short causal convolution -------------------------------------------------------------


def _conv_inputs(x, weight, bias, dims: int, silu: bool):
    torch = _torch()
    code = _tokens(x, dims)
    D, dev = x.shape[-1], x.device
    if weight.dim() != 2:
        raise ValueError("weight is [D, W]")
    W = weight.shape[1]
    _same(weight, "weight", (D, W), torch.float32, dev)
    _maybe(bias, "bias", (D,), torch.float32, dev)
    T = x.shape[1] if dims == 3 else 1
    return ConvDesc(x.shape[0], T, D, W, code, 1 if silu else 0)


def conv_forward(x, weight, bias=None, *, s0=None, lengths=None, silu: bool = False,
                 want_state: bool = False, out=None):
    """The depthwise causal convolution over [B, T, D] (wkv7_conv_forward):
    pre_t = bias + sum_k weight[:, k] x_{t-(W-1)+k} with W = 2, 3 or 4 taps, y_t =
    pre_t or (``silu``) pre_t sigmoid(pre_t).  ``weight`` float32 [D, W], ``bias``
    float32 [D].  ``s0`` [B, W-1, D] holds the inputs before the first token (None:
    zeros).  Returns ``(y, sT)``; ``sT`` (with ``want_state``, else None) holds the
    last W - 1 inputs, for ``conv_step`` or a continued prompt.

    The token shift x_t + mu (x_{t-1} - x_t) is ``weight = stack([mu, 1 - mu], 1)``.
    """
    torch = _torch()
    d = _conv_inputs(x, weight, bias, 3, silu)
    past = (d.B, d.W - 1, d.D)
    _maybe(s0, "s0", past, x.dtype, x.device)
    _maybe(lengths, "lengths", (d.B,), torch.int32, x.device)
    y = _result(out, "out", x, (x, s0, weight, bias, lengths))
    sT = torch.empty(past, device=x.device, dtype=x.dtype) if want_state else None
    _call("wkv7_conv_forward", x.device, ctypes.byref(d), _ptr(weight), _ptr(bias), _ptr(lengths),
          _ptr(x), _ptr(s0), _ptr(y), _ptr(sT))
    return y, sT


def conv_backward(x, weight, dy, bias=None, *, s0=None, dsT=None, lengths=None, silu: bool = False,
                  want_ds0: bool = True, workspace=None):
    """Gradients of ``<dy, y> + <dsT, sT>`` (wkv7_conv_backward): returns ``(dx,
    dweight, dbias, ds0)``; dbias is None without a bias, ds0 without ``want_ds0``."""
    torch = _torch()
    d = _conv_inputs(x, weight, bias, 3, silu)
    past = (d.B, d.W - 1, d.D)
    _same(dy, "dy", x.shape, x.dtype, x.device)
    _maybe(s0, "s0", past, x.dtype, x.device)
    _maybe(dsT, "dsT", past, x.dtype, x.device)
    _maybe(lengths, "lengths", (d.B,), torch.int32, x.device)
    dx, dweight = torch.empty_like(x), torch.empty_like(weight)
    dbias = torch.empty_like(bias) if bias is not None else None
    ds0 = torch.empty(past, device=x.device, dtype=x.dtype) if want_ds0 else None
    ws, wsb, _held = _scratch(workspace, lib().wkv7_conv_backward_workspace_bytes(ctypes.byref(d)), x.device)
    _call("wkv7_conv_backward", x.device, ctypes.byref(d), _ptr(weight), _ptr(bias), _ptr(lengths),
          _ptr(x), _ptr(s0), _ptr(dy), _ptr(dsT), _ptr(dx), _ptr(dweight), _ptr(dbias), _ptr(ds0), ws, wsb)
    return dx, dweight, dbias, ds0


def conv_step(x, weight, state, bias=None, *, silu: bool = False, out=None):
    """One token, x [B, D] (wkv7_conv_step): returns y [B, D] and moves ``state``
    [B, W-1, D] on in place."""
    d = _conv_inputs(x, weight, bias, 2, silu)
    _same(state, "state", (d.B, d.W - 1, d.D), x.dtype, x.device)
    y = _result(out, "out", x, (x, state, weight, bias))
    _call("wkv7_conv_step", x.device, ctypes.byref(d), _ptr(weight), _ptr(bias), _ptr(x), _ptr(state), _ptr(y))
    return y


# ---- the selective scan -----------------------------------------------------------------------


class SsmGrads(NamedTuple):
    """Gradients of ``ssm_backward``; dz, ddskip, ddt_bias, dh0 are None without theirs."""
    dx: object
    ddt: object
    dA: object
    dB: object
    dC: object
    dz: object
    ddskip: object
    ddt_bias: object
    dh0: object


def _ssm_inputs(x, dt, A, Bm, Cm, z, dskip, dt_bias, lengths, dims: int, ckpt_bits: int, softplus: bool):
    torch = _torch()
    code = _tokens(x, dims)
    D, dev, f32 = x.shape[-1], x.device, torch.float32
    _same(dt, "dt", x.shape, x.dtype, dev)
    _maybe(z, "z", x.shape, x.dtype, dev)
    if A.dim() != 2 or Bm.dim() != dims + 1:
        raise ValueError("A is [D, N]; Bm and Cm are the tokens' shape with [G, N] in place of D")
    N, G = A.shape[1], Bm.shape[-2]
    _same(A, "A", (D, N), f32, dev)
    shape = tuple(x.shape[:-1]) + (G, N)
    _same(Bm, "Bm", shape, x.dtype, dev)
    _same(Cm, "Cm", shape, x.dtype, dev)
    _maybe(dskip, "dskip", (D,), f32, dev)
    _maybe(dt_bias, "dt_bias", (D,), f32, dev)
    _maybe(lengths, "lengths", (x.shape[0],), torch.int32, dev)
    desc = SsmDesc(x.shape[0], x.shape[1] if dims == 3 else 1, D, N, G, code, ckpt_bits)
    return desc, SsmParams(_ptr(A), _ptr(dskip), _ptr(dt_bias), _ptr(lengths), 1 if softplus else 0)


def ssm_ckpt_bytes(desc: SsmDesc) -> int:
    return int(lib().wkv7_ssm_ckpt_bytes(ctypes.byref(desc)))


def ssm_split_ckpt(ckpt, B: int, T: int, D: int, N: int):
    """Views of an 8-bit checkpoint: int8 codes [B, ceil(T/16), D, N] and float32
    scales [B, ceil(T/16), D]; a state is code * scale."""
    torch = _torch()
    n = (T + 15) // 16
    size = B * n * D * N
    at = (size + 15) // 16 * 16
    return (ckpt[:size].view(torch.int8).view(B, n, D, N),
            ckpt[at:at + B * n * D * 4].view(torch.float32).view(B, n, D))


def ssm_forward(x, dt, A, Bm, Cm, *, z=None, dskip=None, dt_bias=None, h0=None, lengths=None,
                softplus: bool = True, want_state: bool = True, ckpt_bits: int = 0, out=None, workspace=None):
    """The selective scan over [B, T, D] (wkv7_ssm_forward), per channel d of group g:

        D_t = softplus(dt_t + dt_bias)   (``softplus=False``: dt_t + dt_bias itself)
        h[n] = exp(D_t A[d, n]) h[n] + D_t x_t Bm_t[g, n]
        y_t = (sum_n Cm_t[g, n] h[n] + dskip x_t) z_t sigmoid(z_t)

    ``A`` float32 [D, N] with N = 8, 16, 32 or 64; ``Bm``, ``Cm`` [B, T, G, N] for G
    groups of D / G neighbouring channels; ``z`` [B, T, D], ``dskip``, ``dt_bias``
    float32 [D] may be None; ``h0`` float32 [B, D, N] (None: zeros).

    Returns ``(y, hT, ckpt)``.  ``ckpt_bits`` 32 or 8 keeps the state entering
    every 16 tokens for ``ssm_backward``: float32 [B, ceil(T/16), D, N], or a flat
    uint8 tensor of int8 codes and their scales (``ssm_split_ckpt``), 0.31 of the
    bytes at N = 16.
    """
    torch = _torch()
    d, prm = _ssm_inputs(x, dt, A, Bm, Cm, z, dskip, dt_bias, lengths, 3, ckpt_bits, softplus)
    state = (d.B, d.D, d.N)
    _maybe(h0, "h0", state, torch.float32, x.device)
    y = _result(out, "out", x, (x, dt, Bm, Cm, z, A, dskip, dt_bias, h0, lengths))
    hT = torch.empty(state, device=x.device, dtype=torch.float32) if want_state else None
    ckpt = None
    if ckpt_bits == 32:
        ckpt = torch.empty((d.B, (d.T + 15) // 16, d.D, d.N), device=x.device, dtype=torch.float32)
    elif ckpt_bits:
        ckpt = torch.empty(ssm_ckpt_bytes(d), device=x.device, dtype=torch.uint8)
    ws, wsb, _held = _scratch(workspace, lib().wkv7_ssm_forward_workspace_bytes(ctypes.byref(d)), x.device)
    _call("wkv7_ssm_forward", x.device, ctypes.byref(d), ctypes.byref(prm), _ptr(x), _ptr(dt), _ptr(Bm),
          _ptr(Cm), _ptr(z), _ptr(h0), _ptr(y), _ptr(hT), _ptr(ckpt), ws, wsb)
    return y, hT, ckpt


def ssm_backward(x, dt, A, Bm, Cm, dy, ckpt, *, z=None, dskip=None, dt_bias=None, dhT=None, lengths=None,
                 softplus: bool = True, ckpt_bits: int = 32, want_dh0: bool = True,
                 workspace=None) -> SsmGrads:
    """Gradients of ``<dy, y> + <dhT, hT>`` (wkv7_ssm_backward) from the inputs of
    ``ssm_forward`` and the ``ckpt`` it returned for the same ``ckpt_bits``."""
    torch = _torch()
    if ckpt_bits not in (8, 32):
        raise ValueError("ckpt_bits is 8 or 32")
    d, prm = _ssm_inputs(x, dt, A, Bm, Cm, z, dskip, dt_bias, lengths, 3, ckpt_bits, softplus)
    state, dev, f32 = (d.B, d.D, d.N), x.device, torch.float32
    _same(dy, "dy", x.shape, x.dtype, dev)
    _maybe(dhT, "dhT", state, f32, dev)
    if ckpt_bits == 32:
        _same(ckpt, "ckpt", (d.B, (d.T + 15) // 16, d.D, d.N), f32, dev)
    else:
        _same(ckpt, "ckpt", (ssm_ckpt_bytes(d),), torch.uint8, dev)
    # Without channels the entry point writes nothing, and B and C have gradients all the same.
    shared = torch.empty_like if d.D else torch.zeros_like
    g = SsmGrads(torch.empty_like(x), torch.empty_like(x), torch.empty_like(A), shared(Bm), shared(Cm),
                 None if z is None else torch.empty_like(x),
                 None if dskip is None else torch.empty_like(dskip),
                 None if dt_bias is None else torch.empty_like(dt_bias),
                 torch.empty(state, device=dev, dtype=f32) if want_dh0 else None)
    ptrs = SsmGradPointers(_ptr(g.dx), _ptr(g.ddt), _ptr(g.dB), _ptr(g.dC), _ptr(g.dz), _ptr(g.dA),
                           _ptr(g.ddskip), _ptr(g.ddt_bias), _ptr(g.dh0))
    ws, wsb, _held = _scratch(workspace, lib().wkv7_ssm_backward_workspace_bytes(ctypes.byref(d)), dev)
    _call("wkv7_ssm_backward", dev, ctypes.byref(d), ctypes.byref(prm), _ptr(x), _ptr(dt), _ptr(Bm), _ptr(Cm),
          _ptr(z), _ptr(dy), _ptr(dhT), _ptr(ckpt), ctypes.byref(ptrs), ws, wsb)
    return g


def ssm_step(x, dt, A, Bm, Cm, state, *, z=None, dskip=None, dt_bias=None, softplus: bool = True, out=None):
    """One token, x [B, D], Bm and Cm [B, G, N] (wkv7_ssm_step): returns y [B, D] and
    updates ``state`` [B, D, N] in place."""
    torch = _torch()
    d, prm = _ssm_inputs(x, dt, A, Bm, Cm, z, dskip, dt_bias, None, 2, 0, softplus)
    _same(state, "state", (d.B, d.D, d.N), torch.float32, x.device)
    y = _result(out, "out", x, (x, dt, Bm, Cm, z, state, A, dskip, dt_bias))
    _call("wkv7_ssm_step", x.device, ctypes.byref(d), ctypes.byref(prm), _ptr(x), _ptr(dt), _ptr(Bm), _ptr(Cm),
          _ptr(z), _ptr(state), _ptr(y))
    return y
