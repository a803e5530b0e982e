"""Binding of the gated linear recurrence (kda_gated_scan_*): h_t = a_t h_{t-1}
+ w_t x_t per channel, over whole sequences with its gradient, and one token at
a time. Only arguments are marshalled here."""
import ctypes
import functools

import torch

from . import _lib
from .kda import _DTYPES, _need, _on_stream, _ptr


def _scan_options(gate, gate_lower, write, zero_outside=False):
    """kda_scan_options by reference. The bound counts as the number it is now: a tensor
    would be known again by its identity, whatever it holds."""
    return _options_of(gate, float(gate_lower), write, zero_outside)


@functools.lru_cache(maxsize=64)
def _options_of(gate, gate_lower, write, zero_outside):
    """The options' struct, one for each combination in use."""
    if gate not in _lib.GATE or write not in _lib.WRITE:
        raise ValueError("gate must be one of %s and write one of %s"
                         % (sorted(_lib.GATE), sorted(_lib.WRITE)))
    return ctypes.byref(_lib.ScanOptions(_lib.GATE[gate], gate_lower, _lib.WRITE[write], zero_outside))


def _rows(x, g, lead):
    """Checks x and g, with ``lead`` dimensions before the channels'; returns the
    first of them and the number of channels."""
    _need(x, "x")
    _need(g, "g")
    if x.dtype not in _DTYPES or g.dtype not in _DTYPES:
        raise ValueError("x and g must be bfloat16 or float32")
    shape = x.shape
    if len(shape) <= lead:
        raise ValueError("x must be [%schannels...]" % ("B, T, " if lead == 2 else "N, "))
    if g.shape != shape:
        raise ValueError("g must have x's shape")
    D = 1
    for n in shape[lead:]:
        D *= n
    return shape[0], D


def _tokens(x, g, cu_seqlens):
    """Checks x [B, T, ...], g and cu_seqlens; returns B, T, D, num_seqs."""
    B, D = _rows(x, g, 2)
    T = x.shape[1]
    if cu_seqlens is None:
        return B, T, D, B
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    if B != 1 or cu_seqlens.numel() < 2:
        raise ValueError("packed sequences need B = 1 and cu_seqlens [N + 1]")
    return B, T, D, cu_seqlens.numel() - 1


def _states(t, name, N, x):
    """Checks a states tensor [N, channels...] fp32."""
    _need(t, name, torch.float32)
    if t.shape != (N,) + x.shape[2:]:
        raise ValueError("%s must be [%d, %s]" % (name, N, ", ".join(map(str, x.shape[2:]))))


def _like(t, name, of, what):
    _need(t, name, of.dtype)
    if t.shape != of.shape:
        raise ValueError("%s must have %s's shape" % (name, what))


def _carry_rows(B, T, N):
    return B * T // _lib.SCAN_CARRY_TOKENS + N


def _carries(t, B, T, N, D):
    _need(t, "carries", torch.float32, 2)
    if t.shape != (_carry_rows(B, T, N), D):
        raise ValueError("carries must be [%d, %d]" % (_carry_rows(B, T, N), D))


def gated_scan_fwd(x, g, init_state=None, cu_seqlens=None, *, out=None, final_state=None,
                   carries=None, save_carries=False, output_final_state=True, stream=None,
                   gate="log", gate_lower=-5.0, write="plain"):
    """The gated linear recurrence h_t = a_t h_{t-1} + w_t x_t, per channel, over
    whole sequences (kda_gated_scan_fwd). x [B, T, channels...] (bf16 or fp32;
    the channels in any number of dimensions, e.g. [B, T, H, d]); g of x's shape
    (fp32, or bf16 with bf16 x); init_state [N, channels...] fp32 or None;
    cu_seqlens int32 [N + 1] (device) or None (then N = B). The number of
    channels must be a multiple of 8 (of 4 with fp32 x).
    Returns (out, final_state or None, carries or None): out the states h_t in
    x's type, final_state [N, channels...] fp32.
    ``gate``: "log" (g is log a), "logsigmoid" (a = sigmoid(g)) or "bounded"
    (log a = gate_lower * sigmoid(g)). ``write``: "plain" (w = 1), "complement"
    (w = 1 - a) or "norm" (w = sqrt(1 - a^2)).
    ``save_carries`` (or a ``carries`` buffer) keeps what gated_scan_bwd needs:
    the fp32 state entering every 64th token, [B T // 64 + N, D].
    Rows outside every sequence (before cu_seqlens[0], from cu_seqlens[N] on) are
    zeros in the returned ``out``, and left as they were in one that is given.
    No autograd graph is built: the gradient is gated_scan_bwd's, which a
    torch.autograd.Function of the caller's can call."""
    B, T, D, N = _tokens(x, g, cu_seqlens)
    opts = _scan_options(gate, gate_lower, write, cu_seqlens is not None and out is None)
    if init_state is not None:
        _states(init_state, "init_state", N, x)
    if final_state is not None:
        _states(final_state, "final_state", N, x)
    if out is not None:
        _like(out, "out", x, "x")
    if carries is not None:
        _carries(carries, B, T, N, D)
    return _on_stream(_launch_fwd,
                      ("x", "g", "init_state", "cu_seqlens", "out", "final_state", "carries"),
                      (x, g, init_state, cu_seqlens, out, final_state, carries), stream,
                      x, g, init_state, cu_seqlens, out, final_state, carries, save_carries,
                      output_final_state, B, T, D, N, opts)


def _launch_fwd(x, g, init_state, cu_seqlens, out, final_state, carries, save_carries,
                output_final_state, B, T, D, N, opts, stream):
    if out is None:
        out = torch.empty_like(x)
    if final_state is None and output_final_state:
        final_state = torch.empty((N,) + x.shape[2:], dtype=torch.float32, device=x.device)
    if carries is None and save_carries:
        carries = torch.empty((_carry_rows(B, T, N), D), dtype=torch.float32, device=x.device)
    status = _lib.lib().kda_gated_scan_fwd(
        x.data_ptr(), g.data_ptr(), _ptr(init_state), _ptr(cu_seqlens), out.data_ptr(),
        _ptr(final_state), _ptr(carries), B, T, D, N, _DTYPES[x.dtype], _DTYPES[g.dtype], opts, stream)
    if status:
        _lib.check("kda_gated_scan_fwd", status)
    return out, final_state, carries


def gated_scan_bwd(dout, x, g, carries, cu_seqlens=None, *, dfinal_state=None, dx=None, dg=None,
                   dinit_state=None, output_dinit_state=True, stream=None, gate="log",
                   gate_lower=-5.0, write="plain"):
    """The gradient of gated_scan_fwd (kda_gated_scan_bwd): dout of x's shape and
    type, dfinal_state [N, channels...] fp32 or None; x, g, cu_seqlens and the
    options of the forward call, and the ``carries`` that it saved.
    Returns (dx, dg, dinit_state or None), in the types of x, g and fp32. Rows
    outside every sequence have the gradient zero; in a ``dx`` or ``dg`` that is
    given they are left as they were."""
    B, T, D, N = _tokens(x, g, cu_seqlens)
    opts = _scan_options(gate, gate_lower, write, cu_seqlens is not None and dx is None and dg is None)
    _like(dout, "dout", x, "x")
    _carries(carries, B, T, N, D)
    for t, name in ((dfinal_state, "dfinal_state"), (dinit_state, "dinit_state")):
        if t is not None:
            _states(t, name, N, x)
    if dx is not None:
        _like(dx, "dx", x, "x")
    if dg is not None:
        _like(dg, "dg", g, "g")
    return _on_stream(_launch_bwd,
                      ("x", "g", "dout", "carries", "cu_seqlens", "dfinal_state", "dinit_state", "dx",
                       "dg"),
                      (x, g, dout, carries, cu_seqlens, dfinal_state, dinit_state, dx, dg), stream,
                      dout, x, g, carries, cu_seqlens, dfinal_state, dx, dg, dinit_state,
                      output_dinit_state, B, T, D, N, opts)


def _launch_bwd(dout, x, g, carries, cu_seqlens, dfinal_state, dx, dg, dinit_state,
                output_dinit_state, B, T, D, N, opts, stream):
    # The option zeroes rows in both or in neither; a fresh one beside a given one is
    # zeroed whole.
    fresh = torch.empty_like if cu_seqlens is None or (dx is None and dg is None) else torch.zeros_like
    if dx is None:
        dx = fresh(x)
    if dg is None:
        dg = fresh(g)
    if dinit_state is None and output_dinit_state:
        dinit_state = torch.empty((N,) + x.shape[2:], dtype=torch.float32, device=x.device)
    status = _lib.lib().kda_gated_scan_bwd(
        dout.data_ptr(), _ptr(dfinal_state), x.data_ptr(), g.data_ptr(), carries.data_ptr(),
        _ptr(cu_seqlens), dx.data_ptr(), dg.data_ptr(), _ptr(dinit_state), B, T, D, N,
        _DTYPES[x.dtype], _DTYPES[g.dtype], opts, stream)
    if status:
        _lib.check("kda_gated_scan_bwd", status)
    return dx, dg, dinit_state


def gated_scan_step(x, g, state, *, slots=None, out=None, stream=None, gate="log", gate_lower=-5.0,
                    write="plain"):
    """One token of gated_scan_fwd for N rows, states updated in place
    (kda_gated_scan_step): x, g [N, channels...]; state [N, channels...] fp32,
    or with ``slots`` (int32 [N], on the device) a pool [P, channels...] whose
    slot slots[n] is row n's state. Rows whose slot lies outside [0, P) (-1:
    padding) touch no state and get zeros; slots in range must be distinct.
    Returns out [N, channels...] in x's type. Options as in gated_scan_fwd."""
    N, D = _rows(x, g, 1)
    opts = _scan_options(gate, gate_lower, write)
    _need(state, "state", torch.float32)
    if state.shape[1:] != x.shape[1:]:
        raise ValueError("state must be [slots, %s]" % ", ".join(map(str, x.shape[1:])))
    if slots is None:
        if state.shape[0] != N:
            raise ValueError("state must have one row per row of x, or slots be given")
    else:
        _need(slots, "slots", torch.int32, 1)
        if slots.shape[0] != N:
            raise ValueError("slots must have one entry per row")
    if out is not None:
        _like(out, "out", x, "x")
    return _on_stream(_launch_step, ("x", "g", "state", "slots", "out"), (x, g, state, slots, out), stream,
                      x, g, state, slots, out, N, D, opts)


def _launch_step(x, g, state, slots, out, N, D, opts, stream):
    if out is None:
        out = torch.empty_like(x)
    status = _lib.lib().kda_gated_scan_step(
        x.data_ptr(), g.data_ptr(), state.data_ptr(), _ptr(slots), out.data_ptr(), N, state.shape[0],
        D, _DTYPES[x.dtype], _DTYPES[g.dtype], opts, stream)
    if status:
        _lib.check("kda_gated_scan_step", status)
    return out
