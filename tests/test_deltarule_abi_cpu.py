"""The gated delta rule's and the norm and rotation's entry points without a GPU: workspace queries,
refusals on the host before any device is touched, the frequency table.

Pointers are fake addresses: the library never dereferences a device pointer on the
host, and every call below fails validation."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from xlstm_mlstm_matrix_amd import binding as B

OK, NULL, SHAPE, UNSUP, STATE, WS, ALIAS, HIP, ALIGN = range(9)
M = 1 << 40   # spacing of the fake buffers


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(B.LIB_PATH):
        from xlstm_mlstm_matrix_amd import build
        build.build()
    return B.lib()


def strides(*rows):
    flat = [x for r in rows for x in r]
    return (ctypes.c_longlong * len(flat))(*flat)


def fwd(**kw):
    a = dict(q=M, k=2 * M, v=3 * M, g=4 * M, beta=5 * M, S0=6 * M, lengths=7 * M, o=8 * M, S_T=9 * M, strides=None,
             scale=1.0, B=2, Hk=3, H=6, T=100, dk=64, dv=128, io=1, ws=10 * M, n=1 << 39, stream=None)
    a.update(kw)
    return B.lib().mlstm_deltarule_fwd(*a.values())


def step(**kw):
    a = dict(q=M, k=2 * M, v=3 * M, g=4 * M, beta=5 * M, S=6 * M, o=8 * M, S_out=9 * M, strides=None, scale=1.0,
             B=2, Hk=3, H=6, dk=64, dv=128, io=1, stream=None)
    a.update(kw)
    return B.lib().mlstm_deltarule_step(*a.values())


def bwd(**kw):
    a = dict(q=M, k=2 * M, v=3 * M, g=4 * M, beta=5 * M, S0=6 * M, lengths=7 * M, do=8 * M, dS=9 * M, dq=10 * M,
             gk=11 * M, gv=12 * M, dg=13 * M, db=14 * M, dS0=15 * M, strides=None, scale=1.0, B=2, Hk=3, H=6, T=100,
             dk=64, dv=128, io=1, ws=16 * M, n=1 << 39, stream=None)
    a.update(kw)
    return B.lib().mlstm_deltarule_bwd(*a.values())


@pytest.mark.parametrize("call,need,gates", [(fwd, "q k v o", "g beta"), (step, "q k v o S_out", "g beta"),
                                             (bwd, "q k v do dq gk gv", "g beta dg db")])
def test_deltarule_refusals(call, need, gates):
    for n in need.split():
        assert call(**{n: None}) == NULL, n
        assert call(**{n: M * 20 + 8}) == ALIGN, n
    for n in gates.split():
        assert call(**{n: None}) == NULL, n
        assert call(**{n: M * 20 + 2}) == ALIGN, n
    for n in ("B", "Hk", "H", "dk", "dv"):
        assert call(**{n: 0}) == SHAPE, n
        assert call(**{n: -1}) == SHAPE, n
    assert call(Hk=4) == SHAPE and call(Hk=12) == SHAPE
    assert call(io=2) == UNSUP
    for bad in (dict(dk=8), dict(dk=72), dict(dk=272), dict(dv=24), dict(dv=528)):
        assert call(**bad) == UNSUP, bad
    assert call(B=1 << 16, Hk=1, H=1 << 10) == SHAPE


def test_deltarule_sequence_refusals():
    for call, back in ((fwd, False), (bwd, True)):
        assert call(T=0) == SHAPE and call(T=(1 << 30) + 1, B=1, Hk=1, H=1) == SHAPE
        need = B.deltarule_workspace_size(2, 3, 6, 100, 64, 128, 1, back)
        if need:
            assert call(ws=None) == WS and call(n=need - 1) == WS
    with pytest.raises(B.MlstmError) as e:      # 2^40 bytes
        B.deltarule_workspace_size(1 << 9, 1 << 9, 1 << 9, 1 << 20, 256, 512, 1, True)
    assert e.value.status == SHAPE
    assert fwd(o=M + 16) == ALIAS and fwd(o=4 * M) == ALIAS and fwd(S_T=6 * M + 16) == ALIAS
    assert fwd(S_T=8 * M) == ALIAS and fwd(S_T=5 * M) == ALIAS
    for out in ("dq", "gk", "gv", "dg", "db", "dS0"):
        for at in range(1, 10):
            assert bwd(**{out: at * M}) == ALIAS, (out, at)
    assert bwd(dq=11 * M) == ALIAS and bwd(dg=14 * M) == ALIAS and bwd(dg=15 * M) == ALIAS
    assert step(o=6 * M) == ALIAS and step(S_out=6 * M + 16) == ALIAS and step(S_out=4 * M) == ALIAS


def test_deltarule_strides():
    q, v, g = (3 * 100 * 64, 100 * 64, 64), (6 * 100 * 128, 100 * 128, 128), (600, 100, 1)
    six = lambda q=q, k=q, v=v, g=g, b=g, o=v: strides(q, k, v, g, b, o)
    assert fwd(strides=six(o=(0, 12800, 128))) == ALIAS and fwd(strides=six(q=(-8, 0, 64))) == SHAPE
    assert fwd(strides=six(g=(-1, 100, 1))) == SHAPE and fwd(strides=six(k=(0, 4, 64))) == ALIGN
    assert fwd(strides=six(k=(0, 0, 56))) == SHAPE and fwd(strides=six(k=(0, 0, 1 << 22))) == SHAPE
    assert fwd(strides=six(b=(1 << 62, 0, 1))) == SHAPE
    # a gradient of the gates that repeats values
    assert bwd(strides=strides(q, q, v, g, g, v, q, q, v, (600, 100, 0), g)) == ALIAS


def qk(backward=False, **kw):
    a = dict(q=M, k=2 * M)
    if backward:
        a.update(dyq=3 * M, dyk=4 * M)
    a.update(wq=5 * M, wk=6 * M, f=7 * M, pos=8 * M, yq=9 * M, yk=10 * M)
    if backward:
        a.update(dwq=11 * M, dwk=12 * M)
    a.update(strides=None, B=2, H=4, Hk=2, T=10, d=32, n=8, layout=0, amp=1.0, norm=1, eps=1e-6, io=1)
    if backward:
        a.update(ws=13 * M, wsn=1 << 30)
    a["stream"] = None
    a.update(kw)
    return (B.lib().mlstm_qknorm_bwd if backward else B.lib().mlstm_qknorm_fwd)(*a.values())


@pytest.mark.parametrize("back", [False, True])
def test_qknorm_refusals(back):
    for n in ("q", "yq", "k", "yk", "f") + (("dyq", "dyk") if back else ()):
        assert qk(back, **{n: None}) == NULL, n
    for n in ("wq", "wk", "f", "pos") + (("dwq", "dwk", "ws") if back else ()):
        assert qk(back, **{n: 20 * M + 8}) == ALIGN, n
    assert qk(back, q=M + 1) == ALIGN and qk(back, yk=10 * M + 2, io=0) == ALIGN
    for n in ("B", "H", "Hk", "T", "d"):
        assert qk(back, **{n: 0}) == SHAPE and qk(back, **{n: -3}) == SHAPE
    assert qk(back, n=17) == SHAPE and qk(back, n=-1) == SHAPE
    assert qk(back, d=513, n=0) == UNSUP
    assert qk(back, B=1 << 15, T=1 << 15) == SHAPE
    for n in ("layout", "norm", "io"):
        assert qk(back, **{n: 3}) == UNSUP and qk(back, **{n: -1}) == UNSUP
    assert qk(back, eps=-1.0) == UNSUP and qk(back, eps=float("nan")) == UNSUP
    # results over inputs, tables or one another
    for out in ("yq", "yk"):
        for at in range(5, 9):
            assert qk(back, **{out: at * M}) == ALIAS, (out, at)
    assert qk(back, yq=2 * M) == ALIAS and qk(back, yk=M) == ALIAS and qk(back, yq=10 * M) == ALIAS
    assert qk(back, yq=M + 64) == ALIAS
    s = [(4 * 320, 320, 32), (2 * 320, 320, 32)]
    six = s * (3 if back else 2)
    assert qk(back, strides=strides(*six[:-1], (0, 320, 32))) == ALIAS
    assert qk(back, strides=strides((-32, 0, 0), *six[1:])) == SHAPE
    # heads side by side in fused rows of 6 heads may interleave, heads that meet may not
    row = (10 * 6 * 32, 32, 6 * 32)
    at = dict(yq=9 * M, yk=9 * M + 4 * 32 * 2)
    if back:
        assert qk(True, strides=strides(*s, *s, row, row), ws=None, **at) == WS      # past the overlap rules
    for off in (3 * 32 * 2, 4 * 32 * 2 - 2, 5 * 32 * 2):
        at["yk"] = 9 * M + off
        assert qk(back, strides=strides(*six[:-2], row, row), **at) == ALIAS, off
    # rows at 0, 100, 132 and 232 and those 50 behind them: 132 ... 163 meets 150 ... 181
    odd = dict(T=1, H=2, Hk=2, yq=9 * M, yk=9 * M + 50 * 2)
    dense = [(64, 32, 32)] * (len(six) - 2)
    assert qk(back, strides=strides(*dense, (132, 100, 0), (132, 100, 0)), **odd) == ALIAS
    wider = (10 * 6 * 32, 32, 7 * 32)
    assert qk(back, strides=strides(*six[:-2], row, wider), yq=9 * M, yk=9 * M + 256) == ALIAS
    if back:
        assert qk(True, yq=M) == ALIAS                       # dq over q
        assert qk(True, ws=None) == WS and qk(True, wsn=8) == WS
        for out in ("dwq", "dwk"):
            for at in range(1, 11):
                assert qk(True, **{out: at * M}) == ALIAS, (out, at)
        assert qk(True, dwq=12 * M) == ALIAS and qk(True, dwq=13 * M) == ALIAS


def test_binding_checks():
    t = torch.zeros(1, 1, 2, 16)
    for f in (lambda: B.deltarule_fwd(t, t, t, t, t), lambda: B.qknorm_fwd(t, t), lambda: B.qknorm_bwd(t, t, t, t),
              lambda: B.deltarule_bwd(t, t, t, t, t, t), lambda: B.deltarule_step(t[0], t[0], t[0], t, t)):
        with pytest.raises(ValueError, match="HIP device"):
            f()
    with pytest.raises(TypeError):
        B.deltarule_fwd(None, t, t, t, t)


def test_rope_frequencies():
    n, base = 32, 10000.0
    i = np.arange(n)
    plain, amp = B.rope_frequencies(n)
    exact = base ** (-i / n)
    assert amp == 1.0 and np.allclose(plain.numpy(), exact, rtol=2.0 ** -24, atol=0)
    lin, _ = B.rope_frequencies(n, scaling="linear", factor=4.0)
    assert np.allclose(lin.numpy(), exact / 4, rtol=2.0 ** -24, atol=0)
    big, _ = B.rope_frequencies(n, scaling="base", factor=4.0)
    assert big[0] == 1.0 and np.isclose(big[-1], exact[-1] / 4, rtol=1e-7) and bool((big[1:] < plain[1:]).all())
    ramp, amp = B.rope_frequencies(n, scaling="ramp", factor=4.0, context=4096, fast=32.0, slow=1.0)
    turns = 4096 * exact / (2 * math.pi)
    assert np.isclose(amp, 0.1 * math.log(4.0) + 1.0, rtol=1e-7)
    assert np.allclose(ramp.numpy()[turns >= 32], exact[turns >= 32], rtol=2.0 ** -23, atol=0)
    assert np.allclose(ramp.numpy()[turns <= 1], exact[turns <= 1] / 4, rtol=2.0 ** -23, atol=0)
    between = (turns < 32) & (turns > 1)
    assert between.any() and np.all(ramp.numpy()[between] < exact[between]) and \
        np.all(ramp.numpy()[between] > exact[between] / 4)
    # the ramp is linear in the pair's index
    kept = (ramp.numpy()[between] / exact[between] - 0.25) / 0.75
    assert np.allclose(np.diff(kept, 2), 0, atol=1e-6)


def test_rope_frequencies_refusals():
    f = (ctypes.c_float * 8)()
    a = ctypes.c_float()
    call = lambda n=8, base=1e4, s=0, factor=2.0, ctx=64, fast=32.0, slow=1.0, out=f, amp=ctypes.byref(a): \
        B.lib().mlstm_rope_frequencies(n, base, s, factor, ctx, fast, slow, out, amp)
    assert call() == OK and call(out=None) == NULL and call(amp=None) == NULL
    for bad in (dict(n=0), dict(n=-1), dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")),
                dict(factor=0.5), dict(factor=float("nan")), dict(s=3, ctx=0), dict(s=3, slow=0.0),
                dict(s=3, fast=1.0), dict(s=2, n=1)):
        assert call(**bad) == SHAPE, bad
    assert call(s=4) == UNSUP and call(s=-1) == UNSUP
    with pytest.raises(ValueError):
        B.rope_frequencies(4, scaling="other")
