"""GPU parity of the norm and rotation of queries and keys (qknorm_fwd, qknorm_bwd)
with float64.

Tolerances.  U = 2^-24, a row of d channels with r = 1 / norm.
 * The sum of d squares in float32 is off by at most (d + 1) U of itself, its root by
   half that, the quotient and the products by a few U: z is off by (d / 2 + 8) U |z|.
 * sin and cos: the angle comes within 2^-50 of itself plus 2^-25 of a turn and each is
   off by a few U: 16 U.  y is off by the pair's (|z_a| + |z_b|) A (d / 2 + 8 + 16 + 4) U.
 * dx = r (u w) - x r^3 (sum u w x) / n: (1.5 d + 48) U of the sum of the two terms'
   magnitudes (the second's with all |u w x| added up).
 * dw: N rows in float32, blocks of them first: (d / 2 + 48 + N) U sum |u x r| at the
   most, of which sqrt(N) is what independent roundings reach; 8 sqrt(N) is allowed.
 * A bfloat16 result is rounded once, 2^-8 of itself.
"""
import numpy as np
import pytest
import torch

from oracle import ops as O
from xlstm_mlstm_matrix_amd import binding as B

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24


def close(x, ref, tol, io, what):
    x = x.detach().double().cpu().numpy()
    assert x.shape == ref.shape and np.all(np.isfinite(x)), what
    tol = tol + (2.0 ** -8 if io == "bf16" else U) * np.abs(ref) + 1e-30
    bad = float((np.abs(x - ref) / tol).max())
    print(f"[qknorm] {what}: {bad:.3f} of the bound", flush=True)
    assert bad <= 1.0, (what, bad)


def make(io, Bn, T, H, Hk, d, n_freq, norm, far, seed=0, weight=True, fused=True):
    r = np.random.default_rng(3000 + seed)
    t = lambda *s: torch.from_numpy(r.normal(0, 1, s).astype(np.float32))
    x = t(Bn, T, H + Hk, d).to(DT[io])
    c = {"q": x[:, :, :H].transpose(1, 2), "k": x[:, :, H:].transpose(1, 2)}
    if not fused:
        c = {n: v.contiguous() for n, v in c.items()}
    c["dyq"], c["dyk"] = t(Bn, H, T, d).to(DT[io]), t(Bn, Hk, T, d).to(DT[io])
    c["wq"], c["wk"] = (1 + 0.3 * t(d), 1 + 0.3 * t(d)) if weight else (None, None)
    c["f"] = B.rope_frequencies(n_freq, 1e4)[0] if n_freq else None
    c["pos"] = torch.from_numpy(r.integers(-far, far + 1, (Bn, T)).astype(np.int32)) if far and n_freq else None
    return c


def reference(c, norm, eps, layout, amp):
    """Values and tolerances of (yq, yk), (dq, dk), (dwq, dwk), without the last rounding."""
    y, dx, dw = [], [], []
    kw = dict(inv_freq=c["f"], positions=c["pos"], layout=layout, amp=amp)
    for x, w, dy in ((c["q"], c["wq"], c["dyq"]), (c["k"], c["wk"], c["dyk"])):
        d = x.shape[-1]
        X = O._np(x)
        W = np.ones(d) if w is None else O._np(w)
        r = O._qk_scale(X, norm, eps)
        angle = O._qk_angle(X, c["f"], c["pos"])
        pair = lambda z: np.maximum(np.abs(O._qk_turn(np.abs(z), 0 * angle + np.pi / 4, amp * 2 ** 0.5, layout, 1.0)),
                                    np.abs(O._qk_turn(np.abs(z), 0 * angle + np.pi / 4, amp * 2 ** 0.5, layout, -1.0)))
        n = angle.shape[-1]
        y.append((O.qknorm_forward(x, w, norm, eps, **kw), (d / 2 + 28) * U * pair(X * r * W)))
        g, gw = O.qknorm_backward(x, dy, w, norm, eps, **kw)
        u = pair(O._np(dy))
        terms = r * u * np.abs(W)
        if norm != "none":
            terms = terms + r ** 3 * np.abs(X) * (u * np.abs(W * X)).sum(-1, keepdims=True) / (d if norm == "rms" else 1)
        dx.append((g, (1.5 * d + 48) * U * terms))
        N = X.shape[0] * X.shape[1] * X.shape[2]
        dw.append((gw, (d / 2 + 48 + 8 * N ** 0.5) * U * (u * np.abs(X) * r).sum((0, 1, 2))))
    return y, dx, dw


def run(io, shape, n_freq=0, norm="rms", layout="half", far=0, eps=1e-6, amp=1.0, seed=0, weight=True, fused=True):
    what = f"{io} {shape} n {n_freq} {norm} {layout} far {far} amp {amp}"
    print(f"[qknorm] {what}", flush=True)
    c = make(io, *shape, n_freq, norm, far, seed, weight, fused)
    y, dx, dw = reference(c, norm, eps, layout, amp)
    g = {n: None if t is None else (t.cuda() if n not in "qk" else t.transpose(1, 2).cuda().transpose(1, 2))
         for n, t in c.items()}
    if fused:
        x = torch.cat([g["q"].transpose(1, 2), g["k"].transpose(1, 2)], 2)
        H = g["q"].shape[1]
        g["q"], g["k"] = x[:, :, :H].transpose(1, 2), x[:, :, H:].transpose(1, 2)
    kw = dict(norm=norm, eps=eps, inv_freq=g["f"], positions=g["pos"], layout=layout, amplitude=amp)
    yq, yk = B.qknorm_fwd(g["q"], g["k"], g["wq"], g["wk"], **kw)
    dq, dk, dwq, dwk = B.qknorm_bwd(g["q"], g["k"], g["dyq"], g["dyk"], g["wq"], g["wk"], **kw)
    torch.cuda.synchronize()
    for n, x, (ref, tol) in zip(("yq", "yk", "dq", "dk"), (yq, yk, dq, dk), y + dx):
        close(x, ref, tol, io, f"{what} {n}")
    for n, x, (ref, tol) in zip(("dwq", "dwk"), (dwq, dwk), dw):
        close(x, ref, tol, "f32", f"{what} {n}")
    return g, kw, (yq, yk, dq, dk, dwq, dwk)


SHAPES = [  # B, T, H, Hk, d, n_freq
    (1, 1, 1, 1, 1, 0), (2, 3, 2, 1, 2, 1), (1, 5, 3, 3, 7, 3), (2, 33, 4, 2, 16, 8), (1, 70, 2, 2, 30, 6),
    (3, 17, 8, 2, 64, 32), (1, 130, 4, 4, 128, 64), (2, 40, 10, 5, 96, 36), (1, 9, 2, 1, 200, 100),
    (1, 65, 3, 1, 256, 32), (1, 20, 1, 2, 257, 127), (1, 12, 2, 2, 512, 256), (1, 7, 1, 1, 511, 255),
    (1, 6, 1, 1, 511, 1), (64, 1, 8, 2, 128, 16), (5, 1, 40, 8, 96, 16),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("norm,layout", [("rms", "half"), ("l2", "pairs"), ("none", "half"), ("rms", "pairs")])
def test_shapes(io, shape, norm, layout):
    run(io, shape[:5], shape[5], norm, layout, far=5000, amp=1.25, seed=sum(shape), weight=norm != "l2",
        fused=bool(shape[1] % 2))


@pytest.mark.parametrize("far", [0, 10 ** 6, 2 ** 31 - 1])
def test_far_positions(far):
    """Up to the ends of int32: the product with a float32 frequency has 55 bits, of
    which 53 go on: 2^-22 radians at the very end, within the bound's 16 U only up
    to 2^28, so the last case runs with frequencies of a power of two."""
    c = make("f32", 2, 50, 2, 1, 32, 16, "none", far or 1, 1, False)
    if far > 2 ** 28:
        c["f"] = 2.0 ** -torch.arange(16, dtype=torch.float32)
    if far == 0:
        c["pos"] = None
    y, _, _ = reference(c, "none", 0.0, "half", 1.0)
    g = {n: None if t is None else t.cuda() for n, t in c.items()}
    got = B.qknorm_fwd(g["q"], g["k"], norm="none", inv_freq=g["f"], positions=g["pos"])
    torch.cuda.synchronize()
    for x, (ref, tol) in zip(got, y):
        close(x, ref, tol, "f32", f"far {far}")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 33])
def test_in_place_and_alone(io, d):
    g, kw, out = run(io, (2, 21, 4, 2, d), 8, "rms", "pairs", far=100, seed=3)
    yq, yk, dq, dk, dwq, dwk = out
    alone = B.qknorm_fwd(g["q"], None, g["wq"], **kw)
    assert torch.equal(alone, yq)
    one = B.qknorm_bwd(g["q"], None, g["dyq"], None, g["wq"], **kw)
    assert torch.equal(one[0], dq) and one[1] is None and one[3] is None
    # the sum over rows goes by the sizes, so it may group them differently with keys
    assert torch.allclose(one[2], dwq, rtol=0, atol=float(dwq.abs().max()) * 1e-4)
    none = B.qknorm_bwd(g["q"], g["k"], g["dyq"], g["dyk"], g["wq"], g["wk"], weight_grad=False, **kw)
    assert torch.equal(none[0], dq) and torch.equal(none[1], dk) and none[2] is None
    B.qknorm_bwd(g["q"], g["k"], g["dyq"], g["dyk"], g["wq"], g["wk"], dq=g["dyq"], dk=g["dyk"], **kw)
    B.qknorm_fwd(g["q"], g["k"], g["wq"], g["wk"], yq=g["q"], yk=g["k"], **kw)
    torch.cuda.synchronize()
    for x, y in ((g["dyq"], dq), (g["dyk"], dk), (g["q"], yq), (g["k"], yk)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_rows_of_zeros(io):
    """eps keeps a row of zeros, its gradients are finite."""
    c = make(io, 1, 4, 2, 2, 32, 8, "l2", 10)
    g = {n: None if t is None else t.cuda() for n, t in c.items()}
    g["q"] = torch.zeros_like(g["q"])
    for norm in ("rms", "l2"):
        yq, _ = B.qknorm_fwd(g["q"], g["k"], norm=norm, eps=1e-6, inv_freq=g["f"], positions=g["pos"])
        dq, _, dwq, _ = B.qknorm_bwd(g["q"], g["k"], g["dyq"], g["dyk"], norm=norm, eps=1e-6, inv_freq=g["f"],
                                     positions=g["pos"])
        assert bool((yq == 0).all()) and bool(torch.isfinite(dq).all()) and bool((dwq == 0).all())
        # 1 / sqrt(eps) times the gradient turned back
        ref, _ = O.qknorm_backward(torch.zeros_like(c["q"]), c["dyq"], None, norm, 1e-6, c["f"], c["pos"])
        close(dq, ref, 64 * U * np.abs(ref).max(), io, f"{io} zeros {norm}")


def test_same_bits_twice():
    """Weight gradients of many rows: no order that changes from call to call."""
    c = make("bf16", 4, 700, 6, 3, 128, 64, "rms", 100)
    g = {n: None if t is None else t.cuda() for n, t in c.items()}
    call = lambda: B.qknorm_bwd(g["q"], g["k"], g["dyq"], g["dyk"], g["wq"], g["wk"], inv_freq=g["f"],
                                positions=g["pos"])
    first = call()
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(first, call()))


def test_queries_and_keys_into_the_delta_rule():
    """Projection rows -> unit queries and keys -> delta rule -> head norm, and all
    gradients back, against the oracles chained the same way (float32)."""
    r = np.random.default_rng(5)
    t = lambda *s: torch.from_numpy(r.normal(0, 1, s).astype(np.float32))
    x, v, dy = t(2, 45, 6, 32), t(2, 4, 45, 48), t(2, 45, 4, 48)
    gate, beta = -torch.rand(2, 4, 45) * 0.3, torch.rand(2, 4, 45)
    w, f = 1 + 0.2 * t(4, 48), B.rope_frequencies(8)[0]
    q, k = x[:, :, :2].transpose(1, 2), x[:, :, 2:4].transpose(1, 2)
    c = lambda *xs: [y.cuda() for y in xs]
    gq, gk, gv, gdy, gg, gb, gw, gf = c(q, k, v, dy, gate, beta, w, f)
    kw = dict(norm="l2", eps=1e-6)
    uq, uk = B.qknorm_fwd(gq, gk, inv_freq=gf, **kw)
    o, S = B.deltarule_fwd(uq, uk, gv, gg, gb, scale=0.5)
    y, mean, rstd = B.groupnorm_fwd(o.transpose(1, 2), gw, act="silu")
    do, dw, _ = B.groupnorm_bwd(o.transpose(1, 2), gdy, mean, rstd, gw, act="silu")
    duq, duk, dv, dg, db = B.deltarule_bwd(uq, uk, gv, gg, gb, do.transpose(1, 2), scale=0.5)
    dq, dk, _, _ = B.qknorm_bwd(gq, gk, duq, duk, weight_grad=False, inv_freq=gf, **kw)
    torch.cuda.synchronize()
    ok = dict(norm="l2", eps=1e-6, inv_freq=f)
    ruq, ruk = O.qknorm_forward(q, **ok), O.qknorm_forward(k, **ok)
    ro, _ = O.deltarule_forward(ruq, ruk, v, gate, beta, None, None, 0.5)
    ry, rm, rr = O.groupnorm_forward(ro.transpose(0, 2, 1, 3), w, None, 1e-5, "silu", "token")
    rdo, rdw, _ = O.groupnorm_backward(ro.transpose(0, 2, 1, 3), dy, rm, rr, w, None, "silu", "token")
    rd = O.deltarule_backward(ruq, ruk, v, gate, beta, rdo.transpose(0, 2, 1, 3), None, None, None, 0.5)
    rq, _ = O.qknorm_backward(q, rd[0], None, "l2", 1e-6, f)
    rk, _ = O.qknorm_backward(k, rd[1], None, "l2", 1e-6, f)
    for n, a, b in (("y", y, ry), ("dw", dw, rdw), ("dv", dv, rd[2]), ("dg", dg, rd[3]), ("db", db, rd[4]),
                    ("dq", dq, rq), ("dk", dk, rk)):
        err = np.abs(a.double().cpu().numpy() - b).max() / np.abs(b).max()
        print(f"[qknorm] chain {n}: {err:.2e}", flush=True)
        # sums of at most 256 terms in a row, each operator's own about eight times over, the head
        # norm's 1 / std of small outputs (up to 10) on top: 256 * 8 * 10 U
        assert err <= 256 * 8 * 10 * U, n
