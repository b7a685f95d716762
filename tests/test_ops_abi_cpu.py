"""The C ABI of include/mlstm_ops.h without a GPU: exports, workspace queries,
and refusals on the host before any device is touched.

Pointers are fake addresses: the library never dereferences a pointer on the
host, and every call below fails validation."""
import ctypes
import os
import re
import subprocess

import pytest

from xlstm_mlstm_matrix_amd import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, UNSUP, STATE, WS, ALIAS, HIP, ALIGN = range(9)
M = 1 << 40   # spacing of the fake buffers


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(B.LIB_PATH):
        from xlstm_mlstm_matrix_amd import build
        build.build()
    return B.lib()


def test_exports_every_declared_function(lib):
    with open(os.path.join(ROOT, "include", "mlstm_ops.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"\b(mlstm_[a-z_0-9]+)\s*\(", text))
    assert names == set(B.OPS_SIGNATURES)
    out = subprocess.run(["nm", "-D", "--defined-only", B.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert names <= set(re.findall(r"\sT\s+(mlstm_\w+)", out))


def strides(*rows):
    flat = [x for r in rows for x in r]
    return (ctypes.c_longlong * len(flat))(*flat)


def fwd(**kw):
    a = dict(q=M, k=2 * M, v=3 * M, g=4 * M, S0=5 * M, lengths=6 * M, o=7 * M, S_T=8 * M, strides=None,
             scale=1.0, B=2, H=3, T=100, dk=64, dv=128, io=1, ws=9 * M, n=1 << 36, stream=None)
    a.update(kw)
    return B.lib().mlstm_linattn_fwd(*a.values())


def step(**kw):
    a = dict(q=M, k=2 * M, v=3 * M, g=4 * M, S=5 * M, o=7 * M, S_out=8 * M, strides=None, scale=1.0, B=2, H=3,
             dk=64, dv=128, io=1, stream=None)
    a.update(kw)
    return B.lib().mlstm_linattn_step(*a.values())


def bwd(**kw):
    a = dict(q=M, k=2 * M, v=3 * M, g=4 * M, S0=5 * M, lengths=6 * M, do=7 * M, dS=8 * M, dq=9 * M, gk=10 * M,
             gv=11 * M, dS0=12 * M, strides=None, scale=1.0, B=2, H=3, T=100, dk=64, dv=128, io=1, ws=13 * M,
             n=1 << 36, stream=None)
    a.update(kw)
    return B.lib().mlstm_linattn_bwd(*a.values())


@pytest.mark.parametrize("call,need", [(fwd, "q k v g o"), (step, "q k v g o S_out"),
                                       (bwd, "q k v g do dq gk gv")])
def test_linattn_common_refusals(call, need):
    for n in need.split():
        assert call(**{n: None}) == NULL, n
        assert call(**{n: M * 20 + 8}) == ALIGN, n
    for n in ("B", "H", "dk", "dv"):
        assert call(**{n: 0}) == SHAPE, n
        assert call(**{n: -1}) == SHAPE, n
    assert call(io=2) == UNSUP
    for bad in (dict(dk=8), dict(dk=72), dict(dk=272), dict(dv=24), dict(dv=528)):
        assert call(**bad) == UNSUP, bad
    assert call(B=1 << 16, H=1 << 10) == SHAPE


def test_linattn_fwd_refusals():
    assert fwd(T=0) == SHAPE
    assert fwd(T=(1 << 30) + 1, B=1, H=1) == SHAPE and bwd(T=(1 << 30) + 1, B=1, H=1) == SHAPE
    need = B.linattn_workspace_size(2, 3, 100, 64, 128, 1)
    if need:
        assert fwd(ws=None) == WS and fwd(n=need - 1) == WS
    # o over an input, S_T partly over S0, o over S_T
    assert fwd(o=M + 16) == ALIAS
    assert fwd(S_T=5 * M + 16) == ALIAS
    assert fwd(S_T=7 * M) == ALIAS
    assert fwd(S_T=4 * M) == ALIAS


def test_linattn_strides():
    q, v = (3 * 100 * 64, 100 * 64, 64), (3 * 100 * 128, 100 * 128, 128)
    assert fwd(strides=strides(q, q, v, (0, 100 * 128, 128))) == ALIAS       # o repeats over b
    assert fwd(strides=strides(q, q, v, (3 * 100 * 128, 64, 128))) == ALIAS  # o's heads overlap
    assert fwd(strides=strides(q, q, (-8, 0, 128), v)) == SHAPE              # negative
    assert fwd(strides=strides(q, q, (0, 4, 128), v)) == ALIGN
    assert fwd(strides=strides(q, (0, 0, 56), v, v)) == SHAPE                # rows overlap
    assert fwd(strides=strides(q, (0, 0, 1 << 22), v, v)) == SHAPE
    assert fwd(strides=strides(q, (1 << 62, 0, 64), v, v)) == SHAPE
    # dv interleaved with dk in one buffer: their extents overlap
    t = (100 * 6 * 64, 64, 6 * 64)
    tv = (3 * 100 * 128, 100 * 128, 128)
    assert bwd(strides=strides(q, q, tv, tv, t, t, tv), gk=9 * M + 3 * 64 * 2) == ALIAS


def test_linattn_bwd_refusals():
    assert bwd(T=0) == SHAPE
    need = B.linattn_workspace_size(2, 3, 100, 64, 128, 1, True)
    if need:
        assert bwd(ws=None) == WS and bwd(n=need - 1) == WS
    for out in ("dq", "gk", "gv", "dS0"):
        for at in (1, 2, 3, 4, 5, 6, 7, 8):
            assert bwd(**{out: at * M}) == ALIAS, (out, at)
    assert bwd(dq=10 * M) == ALIAS


def test_linattn_step_refusals():
    assert step(o=M) == ALIAS
    assert step(S_out=5 * M + 16) == ALIAS
    assert step(strides=strides((64, 4, 0), (64, 64, 0), (128, 128, 0), (384, 128, 0))) == ALIGN


def gn_fwd(**kw):
    a = dict(x=M, w=2 * M, b=3 * M, y=4 * M, mean=5 * M, rstd=6 * M, strides=None, N=2, S=10, G=3, D=20, over=1,
             act=1, eps=1e-5, io=1, ws=7 * M, n=1 << 36, stream=None)
    a.update(kw)
    return B.lib().mlstm_groupnorm_fwd(*a.values())


def gn_bwd(**kw):
    a = dict(x=M, dy=2 * M, mean=3 * M, rstd=4 * M, w=5 * M, b=6 * M, dx=7 * M, dw=8 * M, db=9 * M, strides=None,
             N=2, S=10, G=3, D=20, over=1, act=1, io=1, ws=10 * M, n=1 << 36, stream=None)
    a.update(kw)
    return B.lib().mlstm_groupnorm_bwd(*a.values())


def test_groupnorm_refusals():
    for n in ("x", "y", "mean", "rstd"):
        assert gn_fwd(**{n: None}) == NULL, n
    for n in ("x", "dy", "mean", "rstd", "dx"):
        assert gn_bwd(**{n: None}) == NULL, n
    for call in (gn_fwd, gn_bwd):
        for n in ("N", "S", "G", "D"):
            assert call(**{n: 0}) == SHAPE
        assert call(io=5) == UNSUP and call(act=3) == UNSUP and call(over=2) == UNSUP
        assert call(x=M + 2) == ALIGN
        assert call(ws=None, S=4000) == WS
        assert call(G=1 << 20, D=1 << 12) == SHAPE
        assert call(N=1 << 20, S=1 << 12) == SHAPE
    for eps in (0.0, -1.0, float("nan")):
        assert gn_fwd(eps=eps) == UNSUP
    assert gn_fwd(y=M) == ALIAS
    assert gn_fwd(mean=6 * M) == ALIAS
    assert gn_bwd(dx=2 * M) == ALIAS and gn_bwd(dw=9 * M) == ALIAS
    assert gn_fwd(strides=strides((600, 60, 20), (600, 20, 20))) == ALIAS
    assert gn_fwd(strides=strides((600, 60, 20), (0, 60, 20))) == ALIAS
    assert gn_fwd(strides=strides((600, -60, 20), (600, 60, 20))) == SHAPE


def test_workspace_queries():
    n = ctypes.c_size_t(77)
    assert B.lib().mlstm_linattn_fwd_workspace_size(2, 3, 100, 64, 128, 1, None) == NULL
    assert B.lib().mlstm_linattn_fwd_workspace_size(2, 0, 100, 64, 128, 1, ctypes.byref(n)) == SHAPE
    assert B.lib().mlstm_linattn_bwd_workspace_size(2, 3, 100, 65, 128, 1, ctypes.byref(n)) == UNSUP
    assert B.lib().mlstm_groupnorm_workspace_size(2, 3, 4, 0, 0, 1, 0, ctypes.byref(n)) == SHAPE
    assert n.value == 77
    assert B.groupnorm_workspace_size(2, 10, 3, 20, "sequence", B.BF16, True) > 0
    assert B.groupnorm_workspace_size(2, 10, 3, 20, "sequence", B.BF16) == 0       # a workgroup holds a group
    assert B.groupnorm_workspace_size(2, 4000, 3, 20, "sequence", B.BF16) > 0
    assert B.groupnorm_workspace_size(2, 4000, 3, 64, "token", B.BF16) == 0
    with pytest.raises(ValueError):
        B.groupnorm_workspace_size(2, 10, 3, 20, "batch", B.BF16)


def test_binding_refuses_host_tensors_and_types():
    import torch
    z = torch.zeros
    q = z(1, 2, 3, 16)
    for call in (lambda: B.linattn_fwd(q, q, q, z(2)), lambda: B.linattn_bwd(q, q, q, z(2), q),
                 lambda: B.linattn_step(q[:, :, 0], q[:, :, 0], q[:, :, 0], z(2)),
                 lambda: B.groupnorm_fwd(q), lambda: B.groupnorm_bwd(q, q, q, q)):
        with pytest.raises(ValueError, match="HIP device"):
            call()
    with pytest.raises(TypeError):
        B.linattn_fwd([1], q, q, z(2))
