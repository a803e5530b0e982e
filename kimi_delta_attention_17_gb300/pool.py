"""Binding of the state pool's maintenance (kda_state_copy, kda_state_compact).
A pool is a tensor of slots, one per sequence: [P, ...] as decode_step and
gated_scan_step take it with ``slots``, or [L, P, ...] over L layers."""
import torch

from . import _lib
from .kda import _need, _on_stream, _ptr


def _pool(t, name, slot_dim):
    """Checks a pool; returns (layers, slots, bytes per slot)."""
    _need(t, name)
    if slot_dim != 0 and slot_dim != 1:
        raise ValueError("slot_dim must be 0 (a pool [P, ...]) or 1 ([L, P, ...])")
    shape, size = t.shape, t.numel()
    if len(shape) < slot_dim + 2:
        raise ValueError("%s must be [%sP, ...]" % (name, "L, " if slot_dim else ""))
    if size == 0:
        raise ValueError("%s must not be empty" % name)
    layers, slots = shape[0] if slot_dim else 1, shape[slot_dim]
    return layers, slots, t.element_size() * (size // (layers * slots))


def state_copy(pool, src, dst, *, source=None, slot_dim=0, stream=None):
    """pool[dst[i]] = source[src[i]] for every entry i, in place, as one parallel
    assignment (kda_state_copy): all sources are read before any slot is
    written, so beams can be reordered and slots exchanged within one pool.
    One source in several entries forks it; src[i] = -1 clears slot dst[i] to
    zeros; an entry with dst[i] = -1 is skipped, as is one out of range; of
    entries that name one destination the last holds.
    ``pool`` [P, ...] or, with slot_dim=1, [L, P, ...] (every layer alike), any
    type, contiguous, a slot being a multiple of 16 bytes; ``src``, ``dst``
    int32 [n] on the device, n <= 4096; ``source``: another pool of the same
    slots (e.g. chunk_fwd's final_state), or None for ``pool`` itself. Returns
    ``pool``."""
    layers, slots, nbytes = _pool(pool, "pool", slot_dim)
    _need(src, "src", torch.int32, 1)
    _need(dst, "dst", torch.int32, 1)
    if src.shape != dst.shape:
        raise ValueError("src and dst must have the same length")
    source_slots = 0
    if source is not None:
        if source.dtype != pool.dtype or source.dim() != pool.dim():
            raise ValueError("source must have the pool's type and dimensions")
        _, source_slots, _ = _pool(source, "source", slot_dim)
        if source.shape[:slot_dim] + source.shape[slot_dim + 1:] != \
                pool.shape[:slot_dim] + pool.shape[slot_dim + 1:]:
            raise ValueError("source must have the pool's layers and slot shape")
        if source.data_ptr() == pool.data_ptr() and source_slots == slots:
            source = None
    _on_stream(_launch_copy, ("pool", "src", "dst", "source"), (pool, src, dst, source), stream,
               pool, src, dst, source, source_slots, slots, layers, nbytes)
    return pool


def _launch_copy(pool, src, dst, source, source_slots, slots, layers, nbytes, stream):
    status = _lib.lib().kda_state_copy(
        _ptr(source), source_slots, pool.data_ptr(), slots, src.data_ptr(), dst.data_ptr(),
        src.shape[0], layers, nbytes, stream)
    if status:
        _lib.check("kda_state_copy", status)


def state_compact(pool, live, *, slot_dim=0, new_slot=None, count=None, stream=None):
    """Moves the pool's live slots together, in place (kda_state_compact): with n
    live slots, the k-th live slot at or above n moves into the k-th slot below
    n that is not live, so that pool[:n] holds the live states; nothing else is
    written. ``live`` bool or uint8 [P] on the device (not changed); pool and
    slot_dim as in state_copy.
    Returns (new_slot int32 [P]: where each slot's state now is, -1 where it was
    not live; count int32 [1]: n), on the device."""
    layers, slots, nbytes = _pool(pool, "pool", slot_dim)
    _need(live, "live", ndim=1)
    if live.dtype not in (torch.bool, torch.uint8) or live.shape[0] != slots:
        raise ValueError("live must be bool or uint8 [%d]" % slots)
    for t, name, n in ((new_slot, "new_slot", slots), (count, "count", 1)):
        if t is not None:
            _need(t, name, torch.int32, 1)
            if t.shape[0] != n:
                raise ValueError("%s must be int32 [%d]" % (name, n))
    return _on_stream(_launch_compact, ("pool", "live", "new_slot", "count"),
                      (pool, live, new_slot, count), stream,
                      pool, live, new_slot, count, slots, layers, nbytes)


def _launch_compact(pool, live, new_slot, count, slots, layers, nbytes, stream):
    if new_slot is None:
        new_slot = torch.empty(slots, dtype=torch.int32, device=pool.device)
    if count is None:
        count = torch.empty(1, dtype=torch.int32, device=pool.device)
    lib = _lib.lib()
    need = lib.kda_state_compact_workspace_size(slots)
    workspace = torch.empty(need, dtype=torch.uint8, device=pool.device) if need else None
    status = lib.kda_state_compact(
        pool.data_ptr(), slots, live.data_ptr(), new_slot.data_ptr(), count.data_ptr(), layers, nbytes,
        _ptr(workspace), need, stream)
    if status:
        _lib.check("kda_state_compact", status)
    return new_slot, count
