"""Linear attention with one decay per head -- Python binding.

Argument checks and marshalling for the entry points that ``include/wkv7.h``
documents as ``wkv7_linattn_*``.  Token tensors are contiguous float32 or bfloat16
device tensors; states are float32.  All tensors of a call lie on one device; the
work is enqueued on that device's current torch stream.  Outputs may not share
memory with inputs.

Rows of different lengths come padded, tokens [B, T] with ``lengths`` (int32 [B]:
inputs behind a row's length are not used, outputs there are zero), or packed,
tokens [total] with ``starts`` (int32 [B + 1]: row b has the tokens from starts[b]
to starts[b + 1]) and ``max_len``, about the longest row's length; in the tensors that
a call makes, the places of tokens that no row has are zero (a caller's ``out`` keeps
what it held there).
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

from . import LinattnDesc, _dtype_code, _ptr, _torch, lib
from .mixers import _call, _maybe, _result, _same, _scratch


class LinattnGrads(NamedTuple):
    """Gradients of ``linattn_backward``; dg is None with constant decays, ds0 if not wanted."""
    dq: object
    dk: object
    dv: object
    dg: object
    ds0: object


def _inputs(q, k, v, g, lead: int, scale: float):
    """The descriptor for tokens with `lead` leading dimensions, lengths not filled in."""
    torch = _torch()
    code, dev = _dtype_code(v), v.device
    if v.dim() != lead + 2 or q.dim() != lead + 2:
        raise ValueError(f"q, k and v have {lead} leading dimensions, then heads and channels")
    H, P = v.shape[-2:]
    G, N = q.shape[-2:]
    _same(v, "v", v.shape, v.dtype, dev)
    shape = tuple(v.shape[:-2]) + (G, N)
    _same(q, "q", shape, v.dtype, dev)
    _same(k, "k", shape, v.dtype, dev)
    fixed = g.dtype == torch.float32 and g.dim() == 1
    if fixed:
        _same(g, "g", (H,), torch.float32, dev)
    else:
        _same(g, "g", tuple(v.shape[:-1]), v.dtype, dev)
    return LinattnDesc(0, 0, H, G, N, P, code, 1 if fixed else 0, 0, 0, scale)


def _rows(d, v, lengths, starts, max_len):
    """Fills in the rows; returns the pointer to them."""
    torch = _torch()
    if starts is None:
        if max_len is not None:
            raise ValueError("max_len goes with starts")
        d.B, d.T = v.shape[:2]
        return _maybe(lengths, "lengths", (d.B,), torch.int32, v.device)
    if lengths is not None or max_len is None:
        raise ValueError("packed rows take starts and max_len, no lengths")
    if starts.dim() != 1 or starts.shape[0] < 1:
        raise ValueError("starts is [B + 1]")
    _same(starts, "starts", starts.shape, torch.int32, v.device)
    d.B, d.T, d.packed, d.tokens = starts.shape[0] - 1, max_len, 1, v.shape[0]
    return starts


def linattn_ckpt_shape(B: int, T: int, H: int, P: int, N: int, packed_tokens: Optional[int] = None):
    """Shape of the checkpoints: [tiles of 64 tokens, H, P, N]."""
    tiles = B * ((T + 63) // 64) if packed_tokens is None else packed_tokens // 64 + B
    return tiles, H, P, N


def _ckpt_shape(d):
    return linattn_ckpt_shape(d.B, d.T, d.H, d.P, d.N, d.tokens if d.packed else None)


def _clear_rest(d, starts, dev, values, queries=None, keys=None, decays=None):
    """Zeros where the packed call that follows writes nothing."""
    if d.packed:
        _call("wkv7_linattn_clear_rest", dev, ctypes.byref(d), _ptr(starts), _ptr(values), _ptr(queries), _ptr(keys),
              _ptr(decays))


def linattn_forward(q, k, v, g, *, s0=None, lengths=None, starts=None, max_len=None, scale: float = 1.0,
                    want_state: bool = True, want_ckpt: bool = False, out=None, workspace=None):
    """Linear attention (wkv7_linattn_forward), per head h of group h // (H // G), from S = s0:

        S = exp(g_t) S + v_t k_t^T,   y_t = scale S q_t

    ``q``, ``k`` [B, T, G, N] and ``v`` [B, T, H, P] with N and P 32, 64 or 128 (packed:
    [total, ...]); ``g`` [B, T, H] log decays in the tokens' type, or float32 [H],
    constant per head; ``s0`` float32 [B, H, P, N] (None: zeros).

    Returns ``(y, sT, ckpt)``; ``sT`` (with ``want_state``, else None) is the state behind
    each row, ``ckpt`` (with ``want_ckpt``) the states entering every 64 tokens in the
    tokens' type, for ``linattn_backward``.
    """
    torch = _torch()
    d = _inputs(q, k, v, g, 2 if starts is None else 1, scale)
    rows, dev = _rows(d, v, lengths, starts, max_len), v.device
    state = (d.B, d.H, d.P, d.N)
    _maybe(s0, "s0", state, torch.float32, dev)
    y = _result(out, "out", v, (q, k, v, g, s0, rows))
    sT = torch.empty(state, device=dev, dtype=torch.float32) if want_state else None
    ckpt = torch.empty(_ckpt_shape(d), device=dev, dtype=v.dtype) if want_ckpt else None
    ws, wsb, _held = _scratch(workspace, lib().wkv7_linattn_forward_workspace_bytes(ctypes.byref(d)), dev)
    if out is None:
        _clear_rest(d, rows, dev, y)
    _call("wkv7_linattn_forward", dev, ctypes.byref(d), _ptr(rows), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(s0),
          _ptr(y), _ptr(sT), _ptr(ckpt), ws, wsb)
    return y, sT, ckpt


def linattn_backward(q, k, v, g, dy, ckpt, *, dsT=None, lengths=None, starts=None, max_len=None, scale: float = 1.0,
                     want_ds0: bool = True, workspace=None) -> LinattnGrads:
    """Gradients of ``<dy, y> + <dsT, sT>`` (wkv7_linattn_backward) from the inputs of
    ``linattn_forward`` and the ``ckpt`` it returned.  Constant decays have none."""
    torch = _torch()
    d = _inputs(q, k, v, g, 2 if starts is None else 1, scale)
    rows, dev = _rows(d, v, lengths, starts, max_len), v.device
    state = (d.B, d.H, d.P, d.N)
    _same(dy, "dy", v.shape, v.dtype, dev)
    _same(ckpt, "ckpt", _ckpt_shape(d), v.dtype, dev)
    _maybe(dsT, "dsT", state, torch.float32, dev)
    # Without rows or heads the entry point writes nothing.
    new = torch.empty_like if d.B * d.H else torch.zeros_like
    grads = LinattnGrads(new(q), new(k), new(v), None if d.fixed_decay else new(g),
                         torch.empty(state, device=dev, dtype=torch.float32) if want_ds0 else None)
    ws, wsb, _held = _scratch(workspace, lib().wkv7_linattn_backward_workspace_bytes(ctypes.byref(d)), dev)
    _clear_rest(d, rows, dev, grads.dv, grads.dq, grads.dk, grads.dg)
    _call("wkv7_linattn_backward", dev, ctypes.byref(d), _ptr(rows), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(dy),
          _ptr(dsT), _ptr(ckpt), *[_ptr(x) for x in grads], ws, wsb)
    return grads


def linattn_step(q, k, v, g, state, *, slots=None, scale: float = 1.0, out=None):
    """One token (wkv7_linattn_step): q, k [B, G, N], v [B, H, P], g [B, H] or float32 [H].
    Returns y [B, H, P] and updates ``state`` float32 [B, H, P, N] in place; with ``slots``
    (int32 [B]) row b's state is ``state[slots[b]]`` of [slots, H, P, N], and a row whose
    slot does not exist, or is an earlier row's, touches none and gets y = 0."""
    torch = _torch()
    d = _inputs(q, k, v, g, 1, scale)
    d.B, d.T = v.shape[0], 1
    if state.dim() != 4:
        raise ValueError("state is [B or slots, H, P, N]")
    n = d.B if slots is None else state.shape[0]
    _same(state, "state", (n, d.H, d.P, d.N), torch.float32, v.device)
    _maybe(slots, "slots", (d.B,), torch.int32, v.device)
    y = _result(out, "out", v, (q, k, v, g, state, slots))
    _call("wkv7_linattn_step", v.device, ctypes.byref(d), _ptr(slots), n, _ptr(q), _ptr(k), _ptr(v), _ptr(g),
          _ptr(state), _ptr(y))
    return y
