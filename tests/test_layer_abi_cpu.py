"""Refusals of the norms, the 8-bit stores and the decode over several tokens: the C entries check their
arguments before any CUDA call, so these run without a GPU."""
import ctypes

import pytest
import torch

import kimi_delta_attention_17_gb300 as kda
from kimi_delta_attention_17_gb300 import _lib, build

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE = 1 << 20  # 256-byte aligned, never dereferenced on these paths
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


def test_constants_of_the_header():
    text = open(_lib.HEADER).read()
    assert "#define KDA_NORM_SCALE_BLOCK %d\n" % _lib.NORM_SCALE_BLOCK in text
    for name, value in _lib.STORE.items():
        assert "KDA_STORE_%s = %d" % (name.upper(), value) in text


def fwd(L, **kw):
    a = dict(x=FAKE, res=None, w=None, eps=1e-6, out=FAKE + 65536, res_out=None, rstd=None, rows=4, D=12, dt=1, rdt=1)
    a.update(kw)
    return L.kda_rmsnorm_fwd(*a.values(), None)


def quant(L, **kw):
    a = dict(x=FAKE, res=None, w=None, eps=1e-6, out=FAKE + 65536, scales=FAKE, res_out=None, rows=4, D=12, block=128, dt=1, rdt=1)
    a.update(kw)
    return L.kda_rmsnorm_quant(*a.values(), None)


@pytest.mark.parametrize("call", [fwd, quant])
def test_norm_refusals(L, call):
    # D = 12 is the last thing refused: every accepted argument reaches it.
    assert call(L) == UNSUPPORTED
    assert call(L, res=FAKE, res_out=FAKE) == UNSUPPORTED
    for bad in (dict(D=0), dict(D=-8), dict(rows=-1), dict(rows=2 ** 31), dict(dt=2), dict(eps=0.0), dict(eps=-1.0),
                dict(eps=NAN), dict(eps=INF), dict(x=None), dict(res=FAKE), dict(res_out=FAKE), dict(x=FAKE + 8),
                dict(w=FAKE + 4), dict(out=FAKE + 8), dict(res=FAKE + 2, res_out=FAKE), dict(res=FAKE, res_out=FAKE + 8),
                dict(res=FAKE, res_out=FAKE, rdt=3)):
        assert call(L, **bad) == INVALID, bad
    far = FAKE + 4096
    for same in (dict(out=FAKE), dict(res=far, res_out=2 * far, out=far), dict(res=far, res_out=2 * far, out=2 * far)):
        assert call(L, **same) == INVALID, same  # out is what h is or comes from
    assert call(L, res=far, res_out=far) == UNSUPPORTED and call(L, res=far, res_out=FAKE) == UNSUPPORTED
    assert call(L, D=8, out=None) == INVALID
    assert call(L, D=32776) == UNSUPPORTED
    assert call(L, D=8, dt=0, res=FAKE, res_out=FAKE, rdt=1) == UNSUPPORTED
    assert call(L, D=8, rows=0, x=None, out=None) == OK
    if call is quant:
        assert call(L, block=64) == INVALID and call(L, D=8, scales=None) == INVALID
        assert call(L, scales=FAKE + 2) == INVALID
    else:
        assert call(L, rstd=FAKE + 2) == INVALID


def test_norm_gradient_refusals(L):
    def bwd(**kw):
        a = dict(dout=FAKE, h=FAKE, rstd=FAKE, w=FAKE, dh=None, dx=FAKE, dres=None, dw=FAKE, rows=4, D=12, dt=1, hdt=1,
                 ws=FAKE, n=1 << 30)
        a.update(kw)
        return L.kda_rmsnorm_bwd(*a.values(), None)
    assert bwd() == UNSUPPORTED
    for bad in (dict(D=0), dict(rows=-1), dict(rows=2 ** 31), dict(dt=5), dict(hdt=-1), dict(dout=None), dict(h=None),
                dict(rstd=None), dict(dx=None), dict(dout=FAKE + 8), dict(h=FAKE + 8), dict(w=FAKE + 4), dict(dh=FAKE + 8),
                dict(dx=FAKE + 8), dict(dres=FAKE + 8), dict(dres=FAKE), dict(rstd=FAKE + 2), dict(dw=FAKE + 1)):
        assert bwd(**bad) == INVALID, bad
    assert bwd(D=8, dt=0) == UNSUPPORTED
    need = L.kda_rmsnorm_bwd_workspace_size(4000, 8)
    assert 0 < need < 10 ** 6 and L.kda_rmsnorm_bwd_workspace_size(2 ** 31 - 1, 8) < 10 ** 6
    assert L.kda_rmsnorm_bwd_workspace_size(4, 8) == 0 and L.kda_rmsnorm_bwd_workspace_size(0, 8) == 0
    for D in (0, 12, 32776):
        assert L.kda_rmsnorm_bwd_workspace_size(4, D) == 0
    many = dict(D=8, rows=4000)
    assert bwd(**many, ws=None) == WORKSPACE and bwd(**many, n=need - 1) == WORKSPACE and bwd(D=8, ws=FAKE + 64) == WORKSPACE
    assert bwd(D=8, rows=0, dw=None, dout=None, h=None, rstd=None, dx=None, ws=None) == OK


def test_gate_gradient_refusals(L):
    def bwd(**kw):
        a = dict(dout=FAKE, o=FAKE, z=FAKE, w=FAKE, eps=1e-6, do=FAKE, dz=FAKE + 4096, dw=FAKE, tokens=4, H=2, dv=96, dt=1, ws=FAKE,
                 n=1 << 30)
        a.update(kw)
        return L.kda_output_gate_rmsnorm_bwd(*a.values(), None)
    assert bwd() == UNSUPPORTED
    for bad in (dict(tokens=-1), dict(H=0), dict(tokens=2 ** 33), dict(tokens=2 ** 62), dict(dt=2), dict(eps=0.0),
                dict(eps=NAN), dict(dout=None), dict(o=None), dict(z=None), dict(do=None), dict(dz=None), dict(dout=FAKE + 8),
                dict(o=FAKE + 8), dict(z=FAKE + 8), dict(do=FAKE + 8), dict(dz=FAKE + 8), dict(dz=FAKE), dict(w=FAKE + 2), dict(dw=FAKE + 2)):
        assert bwd(**bad) == INVALID, bad
    size = L.kda_output_gate_rmsnorm_bwd_workspace_size
    need = size(4000, 2, 64, 1)
    assert need > 0 and size(4000, 2, 96, 1) == 0 and size(4000, 2, 64, 2) == 0 and size(2 ** 62, 2, 64, 1) == 0
    assert size(4, 2, 64, 1) == 0 and size(2 ** 32, 2, 64, 1) < 10 ** 6
    many = dict(dv=64, tokens=4000)
    assert bwd(**many, ws=None) == WORKSPACE and bwd(**many, n=need - 1) == WORKSPACE and bwd(dv=64, ws=FAKE + 128) == WORKSPACE
    assert bwd(dv=64, tokens=0, dw=None, dout=None, o=None, z=None, do=None, dz=None, ws=None) == OK


@pytest.mark.parametrize("name", ["kda_state_quantize", "kda_state_dequantize"])
def test_store_refusals(L, name):
    far = FAKE + (1 << 40)

    def call(**kw):
        a = dict(pool=FAKE, slots=4, store=far, scales=2 * far, kept=8, src=FAKE, dst=FAKE, n=4097, layers=2, values=256,
                 block=64, format=0)
        a.update(kw)
        if name == "kda_state_dequantize":
            order = ("store", "scales", "kept", "pool", "slots")
            a = {**{x: a[x] for x in order}, **{x: v for x, v in a.items() if x not in order}}
        return getattr(L, name)(*a.values(), None)
    assert call() == UNSUPPORTED  # n, the last thing refused but for the grid
    for bad in (dict(slots=0), dict(kept=0), dict(layers=0), dict(values=0), dict(values=-64), dict(values=250),
                dict(values=2 ** 33), dict(block=16), dict(block=0), dict(block=256), dict(format=2), dict(format=-1),
                dict(n=-1), dict(pool=None), dict(store=None), dict(scales=None), dict(n=1, src=None), dict(n=1, dst=None),
                dict(pool=FAKE + 8), dict(store=far + 8), dict(scales=far + 2), dict(src=FAKE + 2), dict(dst=FAKE + 1),
                dict(store=FAKE + 16), dict(store=FAKE + 4 * 256 * 2 * 4 - 16)):
        assert call(**bad) == INVALID, bad
    assert call(n=4096, layers=65536) == UNSUPPORTED
    assert call(n=0) == OK


def test_decode_tokens_refusals(L):
    def call(**kw):
        a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, scale=1.0, state=FAKE, slots=None, counts=None, out=FAKE, N=2,
                 K=3, P=2, H=2, dk=96, dv=96, dt=1, o=None, write=1)
        a.update(kw)
        return L.kda_decode_tokens(*a.values(), None)
    assert call() == UNSUPPORTED and call(dk=64, dv=128) == UNSUPPORTED
    opts = lambda *o: ctypes.byref(_lib.Options(*o))  # noqa: E731
    for bad in (dict(N=-1), dict(K=-1), dict(H=0), dict(dk=0), dict(dv=-1), dict(P=-1), dict(P=3), dict(slots=FAKE, P=0),
                dict(N=2 ** 16, P=2 ** 16, H=2 ** 15), dict(slots=FAKE, P=2 ** 30), dict(K=2 ** 31 - 1, N=2 ** 12, P=2 ** 12),
                dict(scale=NAN), dict(scale=INF), dict(dt=2), dict(q=None), dict(k=None), dict(v=None), dict(g=None),
                dict(beta=None), dict(state=None), dict(out=None, write=0), dict(q=FAKE + 8), dict(k=FAKE + 8),
                dict(v=FAKE + 8), dict(g=FAKE + 8), dict(state=FAKE + 8), dict(out=FAKE + 8), dict(beta=FAKE + 2),
                dict(slots=FAKE + 2), dict(counts=FAKE + 1), dict(o=opts(3, 0, 0.0, 0)), dict(o=opts(0, 2, 0.0, 0))):
        assert call(**bad) == INVALID, bad
    assert call(g=None, o=opts(2, 0, 0.0, 0)) == UNSUPPORTED and call(g=FAKE + 4, o=opts(1, 0, 0.0, 0)) == UNSUPPORTED
    assert call(out=None) == UNSUPPORTED
    for none in (dict(N=0, P=0), dict(N=0, P=4, slots=FAKE), dict(K=0)):
        assert call(dk=64, dv=64, q=None, k=None, v=None, g=None, beta=None, state=None, out=None, **none) == OK


def test_host_tensors_are_refused():
    x = torch.zeros(2, 8)
    for call in (lambda: kda.rmsnorm_fwd(x), lambda: kda.rmsnorm_quant(x), lambda: kda.rmsnorm_bwd(x, x, x[:, 0]),
                 lambda: kda.output_gate_rmsnorm_bwd(x, x, x), lambda: kda.state_quantize(x, x, x, x, x),
                 lambda: kda.state_dequantize(x, x, x, x, x), lambda: kda.decode_tokens(x, x, x, x, x, 1.0, x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        kda.rmsnorm_fwd([1.0])
