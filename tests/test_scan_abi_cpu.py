"""Refusals of the gated scan, the slot steps and the state pool: the C entries
check their arguments before any CUDA call, and the binding before the C call,
so these run without a GPU."""
import ctypes

import pytest
import torch

from kimi_delta_attention_17_gb300 import (_lib, build, decode_step, gated_scan_bwd, gated_scan_fwd,
                                           gated_scan_step, state_compact, state_copy)

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE = 1 << 20  # 16-byte aligned, never dereferenced on these paths


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


def test_constants_of_the_header():
    text = open(_lib.HEADER).read()
    for name, value in (("KDA_SCAN_CARRY_TOKENS", _lib.SCAN_CARRY_TOKENS),
                        ("KDA_STATE_COPY_MAX", _lib.STATE_COPY_MAX)):
        assert "#define %s %d\n" % (name, value) in text
    for name, value in _lib.WRITE.items():
        assert "KDA_WRITE_%s = %d" % (name.upper(), value) in text


def opts(gate=0, lower=0.0, write=0):
    return ctypes.byref(_lib.ScanOptions(gate, lower, write))


def fwd(L, **kw):
    a = dict(x=FAKE, g=FAKE, init=None, cu=None, out=FAKE, fin=FAKE, car=None, B=1, T=64, D=6, N=1, dt=1,
             gdt=1, o=None)
    a.update(kw)
    return L.kda_gated_scan_fwd(*a.values(), None)


def bwd(L, **kw):
    a = dict(dout=FAKE, dfin=None, x=FAKE, g=FAKE, car=FAKE, cu=None, dx=FAKE, dg=FAKE, dinit=None, B=1,
             T=64, D=6, N=1, dt=1, gdt=1, o=None)
    a.update(kw)
    return L.kda_gated_scan_bwd(*a.values(), None)


@pytest.mark.parametrize("call,tensors", [(fwd, ("x", "g", "out")),
                                          (bwd, ("dout", "x", "g", "car", "dx", "dg"))])
def test_scan_refusals(L, call, tensors):
    # D = 6 is the last thing refused: every accepted argument reaches it.
    assert call(L) == UNSUPPORTED
    for t in tensors:
        assert call(L, **{t: FAKE + 4}) == INVALID
        assert call(L, D=8, **{t: None}) == INVALID
    for bad in (dict(B=0), dict(T=-1), dict(D=0), dict(D=-4), dict(N=0), dict(N=2), dict(dt=2), dict(gdt=-1),
                dict(cu=FAKE, B=2, N=2), dict(cu=FAKE + 2), dict(T=2 ** 31 - 1), dict(B=2 ** 20, T=2 ** 12, N=2 ** 20),
                dict(T=2 ** 22, D=2 ** 18), dict(B=2 ** 19, N=2 ** 19, T=0, D=2 ** 18), dict(o=opts(gate=3)),
                dict(o=opts(write=3)), dict(o=opts(write=-1)), dict(o=opts(gate=2, lower=0.0)),
                dict(o=opts(gate=2, lower=-11.0)), dict(o=opts(gate=2, lower=float("nan")))):
        assert call(L, **bad) == INVALID, bad
    assert call(L, o=opts(gate=2, lower=-5.0, write=2)) == UNSUPPORTED
    assert call(L, cu=FAKE, N=5) == UNSUPPORTED
    assert call(L, D=8, dt=0, gdt=1) == UNSUPPORTED     # fp32 inputs with bf16 gates
    assert call(L, D=12) == UNSUPPORTED                 # bf16 rows of 24 bytes


def test_scan_optional_pointers(L):
    assert fwd(L, init=FAKE + 8) == INVALID and fwd(L, fin=FAKE + 8) == INVALID and fwd(L, car=FAKE + 8) == INVALID
    assert fwd(L, init=None, fin=None) == UNSUPPORTED
    assert bwd(L, dfin=FAKE + 8) == INVALID and bwd(L, dinit=FAKE + 8) == INVALID


def test_carries_size(L):
    f = L.kda_gated_scan_carries_size
    assert f(1, 63, 8, 1) == 32 and f(1, 64, 8, 1) == 64 and f(2, 64, 8, 2) == 128
    assert f(1, 1000, 8, 9) == (1000 // 64 + 9) * 32
    assert f(1, 0, 8, 3) == 96
    for bad in ((0, 1, 8, 1), (1, -1, 8, 1), (1, 1, 0, 1), (1, 1, 8, 0), (2, 1, 8, 3)):
        assert f(*bad) == 0


def test_step_refusals(L):
    def step(**kw):
        a = dict(x=FAKE, g=FAKE, state=FAKE, slots=None, out=FAKE, N=4, P=4, D=6, dt=1, gdt=1, o=None)
        a.update(kw)
        return L.kda_gated_scan_step(*a.values(), None)
    assert step() == UNSUPPORTED
    assert step(slots=FAKE, P=9) == UNSUPPORTED
    assert step(D=8, dt=0, gdt=1) == UNSUPPORTED
    for bad in (dict(x=None), dict(g=None), dict(state=None), dict(out=None), dict(x=FAKE + 8), dict(N=-1),
                dict(P=5), dict(slots=FAKE, P=0), dict(slots=FAKE + 2, P=9), dict(D=0), dict(dt=9), dict(gdt=9),
                dict(o=opts(gate=9)), dict(N=2 ** 30, P=2 ** 30, D=256)):
        assert step(**bad) == INVALID, bad
    assert step(N=0, P=0, D=8, x=None, g=None, state=None, out=None) == OK  # nothing to do


def test_decode_slots_refusals(L):
    def dec(**kw):
        a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, scale=0.1, S=FAKE, slots=FAKE, out=FAKE, N=4, P=8,
                 H=2, dk=96, dv=96, dt=1, o=None)
        a.update(kw)
        return L.kda_decode_step_slots(*a.values(), None)
    assert dec() == UNSUPPORTED
    for bad in (dict(slots=None), dict(slots=FAKE + 2), dict(P=0), dict(P=-1), dict(P=2 ** 30, H=4), dict(S=None),
                dict(N=-1), dict(q=FAKE + 4), dict(scale=float("inf"))):
        assert dec(**bad) == INVALID, bad


def test_pool_refusals(L):
    def copy(**kw):
        a = dict(source=None, sp=0, pool=FAKE, P=4, src=FAKE, dst=FAKE, n=4097, layers=2, nbytes=64)
        a.update(kw)
        return L.kda_state_copy(*a.values(), None)
    assert copy() == UNSUPPORTED                       # one entry too many
    assert copy(n=0, src=None, dst=None) == OK
    far = FAKE + 4 * 2 * 64                            # right behind the pool
    assert copy(source=far, sp=3) == UNSUPPORTED
    assert copy(source=FAKE - 3 * 2 * 64, sp=3) == UNSUPPORTED
    for bad in (dict(pool=None), dict(pool=FAKE + 8), dict(src=None), dict(dst=None), dict(src=FAKE + 2),
                dict(dst=FAKE + 2), dict(n=-1), dict(P=0), dict(layers=0), dict(nbytes=0), dict(nbytes=24),
                dict(nbytes=1 << 35), dict(P=2 ** 30, layers=2 ** 30), dict(source=FAKE + 8, sp=3),
                dict(source=far, sp=0), dict(source=FAKE, sp=4), dict(source=far - 16, sp=3),
                dict(source=FAKE - 3 * 2 * 64 + 16, sp=3)):
        assert copy(**bad) == INVALID, bad

    need = L.kda_state_compact_workspace_size(5000)
    assert need >= 2 * 4 * 5000
    assert [L.kda_state_compact_workspace_size(p) for p in (-1, 0, 1, 4096)] == [0, 0, 0, 0]

    def compact(**kw):
        a = dict(pool=FAKE, P=5000, live=FAKE, new=FAKE, count=FAKE, layers=1, nbytes=64, ws=FAKE, wsb=need - 1)
        a.update(kw)
        return L.kda_state_compact(*a.values(), None)
    assert compact() == WORKSPACE
    assert compact(ws=None, wsb=need) == WORKSPACE
    assert compact(ws=FAKE + 16, wsb=need) == WORKSPACE
    assert compact(P=100, ws=FAKE + 16, wsb=0) == WORKSPACE
    for bad in (dict(pool=None), dict(live=None), dict(new=None), dict(count=None), dict(P=0), dict(layers=-1),
                dict(nbytes=8), dict(pool=FAKE + 4), dict(new=FAKE + 1), dict(count=FAKE + 2)):
        assert compact(**bad) == INVALID, bad


def _cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_before_the_library():
    x, i = _cpu(1, 4, 8), _cpu(4, dtype=torch.int32)
    for call in (lambda: gated_scan_fwd(x, x), lambda: gated_scan_bwd(x, x, x, x),
                 lambda: gated_scan_step(x[0], x[0], x[0]), lambda: state_copy(x, i, i),
                 lambda: state_compact(x, i)):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            call()
    for call in (lambda: gated_scan_fwd(None, x), lambda: gated_scan_step(None, None, None),
                 lambda: state_copy(None, i, i)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError, match="CUDA"):
        decode_step(x, x, x, None, x, 1.0, x, slots=i)
