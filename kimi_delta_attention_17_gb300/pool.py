"""Binding of the state pool's maintenance (kda_state_copy, kda_state_compact) and
of stores that hold states in 8 bits (kda_state_quantize, kda_state_dequantize).
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


_STORE_TYPES = {torch.int8: _lib.STORE["int8"], torch.float8_e4m3fn: _lib.STORE["e4m3"]}


def _store_call(launch, pool, store, scales, src, dst, slot_dim, stream):
    """Checks the arguments of state_quantize and state_dequantize and launches one."""
    _need(pool, "pool", torch.float32)
    _need(store, "store")
    _need(scales, "scales", torch.float32)
    _need(src, "src", torch.int32, 1)
    _need(dst, "dst", torch.int32, 1)
    if slot_dim != 0 and slot_dim != 1:
        raise ValueError("slot_dim must be 0 (a pool [P, ...]) or 1 ([L, P, ...])")
    if store.dtype not in _STORE_TYPES:
        raise ValueError("store must be int8 or float8_e4m3fn")
    shape, kept, factors, lead = pool.shape, store.shape, scales.shape, slot_dim + 1
    if len(shape) <= lead or kept[lead:] != shape[lead:] or (slot_dim and kept[0] != shape[0]) or len(kept) != len(shape):
        raise ValueError("store must have the pool's layers and slot shape")
    if factors[:lead] != kept[:lead]:
        raise ValueError("scales must have the store's layers and slots")
    size, layers = pool.numel(), shape[0] if slot_dim else 1
    if size == 0 or store.numel() == 0:
        raise ValueError("pool and store must not be empty")
    values = size // (layers * shape[slot_dim])
    per = scales.numel() // (layers * kept[slot_dim])
    block = values // per if per and values % per == 0 else 0
    if block not in (32, 64, 128):
        raise ValueError("scales must hold one value for each 32, 64 or 128 of a slot's")
    if src.shape != dst.shape:
        raise ValueError("src and dst must have the same length")
    _on_stream(launch, ("pool", "store", "scales", "src", "dst"), (pool, store, scales, src, dst), stream,
               pool, shape[slot_dim], store, scales, kept[slot_dim], src, dst, layers, values, block)


def _launch_quantize(pool, slots, store, scales, store_slots, src, dst, layers, values, block, stream):
    status = _lib.lib().kda_state_quantize(
        pool.data_ptr(), slots, store.data_ptr(), scales.data_ptr(), store_slots, src.data_ptr(), dst.data_ptr(),
        src.shape[0], layers, values, block, _STORE_TYPES[store.dtype], stream)
    if status:
        _lib.check("kda_state_quantize", status)


def _launch_dequantize(pool, slots, store, scales, store_slots, src, dst, layers, values, block, stream):
    status = _lib.lib().kda_state_dequantize(
        store.data_ptr(), scales.data_ptr(), store_slots, pool.data_ptr(), slots, src.data_ptr(), dst.data_ptr(),
        src.shape[0], layers, values, block, _STORE_TYPES[store.dtype], stream)
    if status:
        _lib.check("kda_state_dequantize", status)


def state_quantize(pool, src, store, scales, dst, *, slot_dim=0, stream=None):
    """store[dst[i]] = pool[src[i]] in 8 bits, for every entry i (kda_state_quantize):
    requests parked, or states of shared prefixes kept, at a quarter of their size.
    ``pool`` fp32 and ``slot_dim`` as in state_copy. ``store`` int8 or float8_e4m3fn:
    [S, ...], or [L, S, ...], with the pool's slot shape. ``scales`` fp32 [S, ...], or
    [L, S, ...]: one for each 32, 64 or 128 consecutive values of a slot, e.g.
    [S, H, dk] for states [S, H, dk, dv] (a scale for each key channel). With m the
    largest magnitude of such a block, a value comes back within m / 254 (int8) or
    2^-4 of itself (e4m3; within m / 458752 near zero).
    ``src``, ``dst`` int32 [n] on the device, n <= 4096, as in state_copy: src -1
    stores zeros, entries out of range are skipped, of entries that name one
    destination the last holds. Returns (store, scales)."""
    _store_call(_launch_quantize, pool, store, scales, src, dst, slot_dim, stream)
    return store, scales


def state_dequantize(store, scales, src, pool, dst, *, slot_dim=0, stream=None):
    """pool[dst[i]] = store[src[i]] as fp32 values, for every entry i
    (kda_state_dequantize): the way back of state_quantize, with its arguments.
    One source in several entries resumes several samples of a prefix. Returns
    ``pool``."""
    _store_call(_launch_dequantize, pool, store, scales, src, dst, slot_dim, stream)
    return pool
