"""Binding of the row norm (kda_rmsnorm_*) and of the output gate's gradient
(kda_output_gate_rmsnorm_bwd). Only arguments are marshalled here."""
import torch

from . import _lib
from .kda import _DTYPES, _need, _on_stream, _ptr


def _rows(x, name):
    """Checks x [..., D]; returns (rows, D)."""
    _need(x, name)
    if x.dtype not in _DTYPES:
        raise ValueError("%s must be bfloat16 or float32" % name)
    shape = x.shape
    if len(shape) == 0 or shape[-1] == 0:
        raise ValueError("%s must be [..., D]" % name)
    return x.numel() // shape[-1], shape[-1]


def _like(t, x, name, dtype=None):
    _need(t, name, dtype)
    if t.shape != x.shape:
        raise ValueError("%s must have the shape %s" % (name, tuple(x.shape)))


def _weight(weight, D, name="weight"):
    if weight is not None:
        _need(weight, name, torch.float32, 1)
        if weight.shape[0] != D:
            raise ValueError("%s must be [%d]" % (name, D))


def _check_sum(x, residual, residual_out, weight):
    """Checks what the norm's forward calls share; returns (rows, D)."""
    rows, D = _rows(x, "x")
    _weight(weight, D)
    if residual is not None:
        _like(residual, x, "residual")
        if residual.dtype != x.dtype and residual.dtype != torch.float32:
            raise ValueError("residual must have x's type or be float32")
        if residual_out is not None:
            _like(residual_out, x, "residual_out", residual.dtype)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    return rows, D


def rmsnorm_fwd(x, weight=None, eps=1e-6, *, residual=None, save_rstd=False, out=None, residual_out=None,
                stream=None):
    """Root-mean-square norm over the last dimension, with the residual's addition
    in front of it (kda_rmsnorm_fwd): h = x + residual, out = weight * h /
    sqrt(mean(h^2) + eps). x [..., D] bf16 or fp32; weight [D] fp32 or None;
    ``residual`` x's shape, of x's type or fp32, or None. h is rounded to the
    residual's type, and what is normalised is that.
    Returns (out, h, rstd): h is ``residual_out`` (which may be ``residual``: in
    place), or x itself without a residual; rstd fp32 x.shape[:-1] with
    ``save_rstd`` (for rmsnorm_bwd), else None. Builds no autograd graph."""
    rows, D = _check_sum(x, residual, residual_out, weight)
    if out is not None:
        _like(out, x, "out", x.dtype)
    return _on_stream(_launch_fwd, ("x", "weight", "residual", "out", "residual_out"),
                      (x, weight, residual, out, residual_out), stream,
                      x, weight, eps, residual, save_rstd, out, residual_out, rows, D)


def _launch_fwd(x, weight, eps, residual, save_rstd, out, residual_out, rows, D, stream):
    if out is None:
        out = torch.empty_like(x)
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(residual)
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device) if save_rstd else None
    status = _lib.lib().kda_rmsnorm_fwd(
        x.data_ptr(), _ptr(residual), _ptr(weight), eps, out.data_ptr(), _ptr(residual_out), _ptr(rstd), rows, D,
        _DTYPES[x.dtype], 0 if residual is None else _DTYPES[residual.dtype], stream)
    if status:
        _lib.check("kda_rmsnorm_fwd", status)
    return out, x if residual is None else residual_out, rstd


def rmsnorm_quant(x, weight=None, eps=1e-6, *, residual=None, scale_per="block", out=None, scales=None,
                  residual_out=None, stream=None):
    """rmsnorm_fwd with its output in 8 bits, for a projection in 8 bits
    (kda_rmsnorm_quant): q = e4m3(y * 448 / m), scale = m / 448 with m the largest
    |y| of a row (``scale_per="row"``) or of 128 values of it ("block"; the last
    block of a row may be a short one). Returns (q float8_e4m3fn [..., D], scales
    fp32 [..., blocks], h); q * scale stands for the output."""
    rows, D = _check_sum(x, residual, residual_out, weight)
    if scale_per != "row" and scale_per != "block":
        raise ValueError('scale_per must be "row" or "block"')
    block = 0 if scale_per == "row" else _lib.NORM_SCALE_BLOCK
    lead = x.shape[:-1] + (-(-D // block) if block else 1,)
    if out is not None:
        _like(out, x, "out", torch.float8_e4m3fn)
    if scales is not None:
        _need(scales, "scales", torch.float32)
        if scales.shape != lead:
            raise ValueError("scales must have the shape %s" % (tuple(lead),))
    return _on_stream(_launch_quant, ("x", "weight", "residual", "out", "scales", "residual_out"),
                      (x, weight, residual, out, scales, residual_out), stream,
                      x, weight, eps, residual, block, out, scales, residual_out, rows, D, lead)


def _launch_quant(x, weight, eps, residual, block, out, scales, residual_out, rows, D, lead, stream):
    if out is None:
        out = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    if scales is None:
        scales = torch.empty(lead, dtype=torch.float32, device=x.device)
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(residual)
    status = _lib.lib().kda_rmsnorm_quant(
        x.data_ptr(), _ptr(residual), _ptr(weight), eps, out.data_ptr(), scales.data_ptr(), _ptr(residual_out), rows, D,
        block, _DTYPES[x.dtype], 0 if residual is None else _DTYPES[residual.dtype], stream)
    if status:
        _lib.check("kda_rmsnorm_quant", status)
    return out, scales, x if residual is None else residual_out


def rmsnorm_bwd(dout, h, rstd, weight=None, *, dh=None, dx=None, dresidual=None, dweight=None, stream=None):
    """Gradient of rmsnorm_fwd (kda_rmsnorm_bwd). dout: gradient of its output, x's
    type; h, rstd: what it returned; ``dh``: the gradient that reaches h from what
    follows (h's type), or None. Returns (dx in dout's type, dresidual in h's type,
    dweight [D] fp32, or None without a weight). Where the two types are the same
    dresidual is dx itself. ``dx`` may be ``dout``, or a ``dh`` of its type, and
    ``dresidual`` may be ``dh`` (in place)."""
    rows, D = _rows(dout, "dout")
    _like(h, dout, "h")
    if h.dtype != dout.dtype and h.dtype != torch.float32:
        raise ValueError("h must have dout's type or be float32")
    _need(rstd, "rstd", torch.float32)
    if rstd.shape != dout.shape[:-1]:
        raise ValueError("rstd must have the shape %s" % (tuple(dout.shape[:-1]),))
    _weight(weight, D)
    _weight(dweight, D, "dweight")
    if dweight is not None and weight is None:
        raise ValueError("dweight needs a weight")
    if dh is not None:
        _like(dh, dout, "dh", h.dtype)
    if dx is not None:
        _like(dx, dout, "dx", dout.dtype)
    if dresidual is not None:
        if h.dtype == dout.dtype:
            raise ValueError("dresidual is dx where h and dout have one type")
        _like(dresidual, dout, "dresidual", h.dtype)
    return _on_stream(_launch_bwd, ("dout", "h", "rstd", "weight", "dh", "dx", "dresidual", "dweight"),
                      (dout, h, rstd, weight, dh, dx, dresidual, dweight), stream,
                      dout, h, rstd, weight, dh, dx, dresidual, dweight, rows, D)


def _launch_bwd(dout, h, rstd, weight, dh, dx, dresidual, dweight, rows, D, stream):
    lib = _lib.lib()
    if dx is None:
        dx = torch.empty_like(dout)
    if dresidual is None and h.dtype != dout.dtype:
        dresidual = torch.empty_like(h)
    need, workspace = 0, None
    if weight is not None:
        if dweight is None:
            dweight = torch.empty_like(weight)
        need = lib.kda_rmsnorm_bwd_workspace_size(rows, D)
        workspace = torch.empty(need, dtype=torch.uint8, device=dout.device) if need else None
    status = lib.kda_rmsnorm_bwd(
        dout.data_ptr(), h.data_ptr(), rstd.data_ptr(), _ptr(weight), _ptr(dh), dx.data_ptr(), _ptr(dresidual),
        _ptr(dweight), rows, D, _DTYPES[dout.dtype], _DTYPES[h.dtype], _ptr(workspace), need, stream)
    if status:
        _lib.check("kda_rmsnorm_bwd", status)
    return dx, dx if dresidual is None else dresidual, dweight


def output_gate_rmsnorm_bwd(dout, o, z, weight=None, eps=1e-6, *, do=None, dz=None, dweight=None, stream=None):
    """Gradient of output_gate_rmsnorm (kda_output_gate_rmsnorm_bwd): dout, o, z
    [..., H, dv] of one dtype; weight and eps as in the forward call. Returns
    (do, dz, dweight [dv] fp32, or None without a weight). ``do`` and ``dz`` may
    each be one of the inputs (in place), but not the same one."""
    _need(o, "o")
    dtype = o.dtype
    if dtype not in _DTYPES:
        raise ValueError("o must be bfloat16 or float32")
    if o.dim() < 2:
        raise ValueError("o must be [..., H, dv]")
    H, dv = o.shape[-2], o.shape[-1]
    for t, name in ((dout, "dout"), (z, "z"), (do, "do"), (dz, "dz")):
        if t is not None or name in ("dout", "z"):
            _like(t, o, name, dtype)
    _weight(weight, dv)
    _weight(dweight, dv, "dweight")
    if dweight is not None and weight is None:
        raise ValueError("dweight needs a weight")
    if H == 0 or dv == 0:
        raise ValueError("o must be [..., H, dv]")
    return _on_stream(_launch_gate_bwd, ("dout", "o", "z", "weight", "do", "dz", "dweight"),
                      (dout, o, z, weight, do, dz, dweight), stream, dout, o, z, weight, eps, do, dz, dweight,
                      o.numel() // (H * dv), H, dv)


def _launch_gate_bwd(dout, o, z, weight, eps, do, dz, dweight, tokens, H, dv, stream):
    lib = _lib.lib()
    if do is None:
        do = torch.empty_like(o)
    if dz is None:
        dz = torch.empty_like(z)
    need, workspace = 0, None
    if weight is not None:
        if dweight is None:
            dweight = torch.empty_like(weight)
        need = lib.kda_output_gate_rmsnorm_bwd_workspace_size(tokens, H, dv, _DTYPES[o.dtype])
        workspace = torch.empty(need, dtype=torch.uint8, device=o.device) if need else None
    status = lib.kda_output_gate_rmsnorm_bwd(
        dout.data_ptr(), o.data_ptr(), z.data_ptr(), _ptr(weight), eps, do.data_ptr(), dz.data_ptr(), _ptr(dweight),
        tokens, H, dv, _DTYPES[o.dtype], _ptr(workspace), need, stream)
    if status:
        _lib.check("kda_output_gate_rmsnorm_bwd", status)
    return do, dz, dweight
