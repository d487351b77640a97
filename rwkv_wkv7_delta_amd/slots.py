"""Slots of a cache of states -- Python binding of the entry points that ``include/wkv7.h``
documents as ``wkv7_slots_*``.

A cache is a contiguous device tensor [planes, slots, ...] of any type (planes: layers; one
with [1, slots, ...], such as ``state[None]``).  Lists of slots are int32 device tensors.
The work is enqueued on the device's current torch stream.
"""

from __future__ import annotations

from . import _ptr, _torch, lib
from .mixers import _call, _same, _scratch


def _cache(t, name: str):
    if t.dim() < 3 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous device tensor [planes, slots, ...]")
    row = t.element_size()
    for n in t.shape[2:]:
        row *= n
    return t.shape[0], t.shape[1], row


def slots_copy(pool, src, dst, *, source=None):
    """In every plane of ``pool``, in order of i: slot dst[i] takes what slot src[i] of
    ``source`` (None: pool itself) holds, or zeros where src[i] is -1 (wkv7_slots_copy).
    Pairs with a slot that does not exist are left out.  Forks, moves and clears states;
    pairs that do not touch each other (free targets, each once) are copied at once."""
    torch = _torch()
    planes, slots, row = _cache(pool, "pool")
    dev = pool.device
    if src.dim() != 1:
        raise ValueError("src and dst are [n]")
    _same(src, "src", src.shape, torch.int32, dev)
    _same(dst, "dst", src.shape, torch.int32, dev)
    read, read_slots = pool, slots
    if source is not None:
        other, read_slots, other_row = _cache(source, "source")
        if other != planes or other_row != row or source.dtype != pool.dtype or source.device != dev:
            raise ValueError("source must have pool's planes, rows, type and device")
        lo, hi = pool.data_ptr(), pool.data_ptr() + pool.numel() * pool.element_size()
        if source.data_ptr() < hi and lo < source.data_ptr() + source.numel() * source.element_size():
            raise ValueError("source overlaps pool")
        read = source
    _call("wkv7_slots_copy", dev, planes, slots, row, src.shape[0], _ptr(src), _ptr(dst), _ptr(read), read_slots,
          _ptr(pool))


def slots_compact(pool, keep, *, clear: bool = False, workspace=None):
    """Moves the slots with ``keep`` (bool or uint8 [slots]) to the front of ``pool``, in
    place in every plane (wkv7_slots_compact): with count of them, those at or behind place
    count fill the free ones before it, in order.  Returns ``(moved, count)``, int32 [slots]
    (a kept slot's new place, else -1) and [1].  What is at or behind place count stays as
    it was, or becomes 0 with ``clear``."""
    torch = _torch()
    planes, slots, row = _cache(pool, "pool")
    dev = pool.device
    if keep.dtype not in (torch.bool, torch.uint8):
        raise ValueError("keep is bool or uint8 [slots]")
    _same(keep, "keep", (slots,), keep.dtype, dev)
    both = torch.empty(slots + 1, device=dev, dtype=torch.int32)
    moved, count = both[:slots], both[slots:]
    ws, wsb, _held = _scratch(workspace, lib().wkv7_slots_compact_workspace_bytes(slots), dev)
    _call("wkv7_slots_compact", dev, planes, slots, row, _ptr(keep), _ptr(moved), _ptr(count), 1 if clear else 0,
          _ptr(pool), ws, wsb)
    return moved, count
