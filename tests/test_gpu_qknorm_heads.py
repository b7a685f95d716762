"""The norm and rotation where a group of lanes walks several heads of a token and a workgroup
takes many turns, forward and backward, against float64 on the device.  Bounds as in
test_gpu_qknorm.py."""
import math

import pytest
import torch

from xlstm_mlstm_matrix_amd import binding as B

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24


def turned(x, angle, amp, layout, sign):
    """Rows [B, H, T, d] with the pairs of their first channels turned by sign * angle [B, T, n]."""
    n = angle.shape[-1]
    if n == 0:
        return x
    c, s = amp * torch.cos(angle)[:, None], sign * amp * torch.sin(angle)[:, None]
    y = x.clone()
    a, b = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def swapped(x, n, layout):
    """The other channel of each pair; zero where there is none."""
    y = torch.zeros_like(x)
    if n:
        a, b = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
        y[..., a], y[..., b] = x[..., b], x[..., a]
    return y


def reference(x, w, dy, angle, norm, eps, amp, layout):
    """Values and bounds (without the last rounding) of y, dx, dw for rows x [B, H, T, d]."""
    d, n = x.shape[-1], angle.shape[-1]
    x, dy = x.double(), dy.double()
    w = torch.ones(d, dtype=torch.float64, device="cuda") if w is None else w.double()
    m = d if norm == "rms" else 1
    r = 1.0 if norm == "none" else 1.0 / torch.sqrt((x * x).sum(-1, keepdim=True) / m + eps)
    # magnitudes of a pair's two terms; sin and cos at their largest
    mag = lambda z: (amp if n else 1.0) * (z.abs() + swapped(z.abs(), n, layout))
    z = x * r * w
    y, ytol = turned(z, angle, amp, layout, 1.0), (d / 2 + 28) * U * mag(z)
    u, au = turned(dy, angle, amp, layout, -1.0), mag(dy)
    dw, dwtol = (u * x * r).sum((0, 1, 2)), (au * x.abs() * r).sum((0, 1, 2))
    dx, terms = r * u * w, r * au * w.abs()
    if norm != "none":
        dx = dx - r ** 3 * x * (u * w * x).sum(-1, keepdim=True) / m
        terms = terms + r ** 3 * x.abs() * (au * (w * x).abs()).sum(-1, keepdim=True) / m
    N = x.shape[0] * x.shape[1] * x.shape[2]
    return (y, ytol), (dx, (1.5 * d + 48) * U * terms), (dw, (d / 2 + 48 + 8 * N ** 0.5) * U * dwtol)


def close(x, ref, half, what):
    ref, tol = ref
    assert x.shape == ref.shape and bool(torch.isfinite(x).all()), what
    bad = float(((x.double() - ref).abs() / (tol + half * ref.abs() + 1e-30)).max())
    print(f"[qknorm] {what}: {bad:.3f} of the bound", flush=True)
    assert bad <= 1.0, (what, bad)


# B, T, H, Hk, d, n_freq: all heads of a token by one group of lanes, some of them with a remainder, more rows
# than one turn of 1024 workgroups, 48 MB and more, a last turn that is not full
SHAPES = [(1, 8200, 5, 2, 128, 64), (3, 1001, 16, 3, 128, 16), (1, 40001, 3, 1, 128, 64), (2, 35001, 2, 1, 128, 32),
          (1, 20001, 15, 4, 128, 0), (3, 1301, 10, 5, 96, 36), (1, 9001, 7, 2, 65, 20), (5, 701, 9, 9, 256, 128),
          (1, 70001, 3, 2, 64, 8), (2, 1503, 6, 4, 511, 100)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("norm,layout", [("rms", "half"), ("l2", "pairs"), ("none", "half")])
def test_many_heads_and_rows(io, shape, norm, layout):
    Bn, T, H, Hk, d, n = shape
    what = f"{io} {shape} {norm} {layout}"
    print(f"[qknorm] {what}", flush=True)
    r = torch.Generator(device="cuda").manual_seed(sum(shape))
    rnd = lambda *s: torch.randn(s, generator=r, device="cuda")
    x = rnd(Bn, T, H + Hk, d).to(DT[io])
    q, k = x[:, :, :H].transpose(1, 2), x[:, :, H:].transpose(1, 2)
    dyq, dyk = rnd(Bn, H, T, d).to(DT[io]), rnd(Bn, Hk, T, d).to(DT[io])
    wq, wk = (1 + 0.3 * rnd(d), 1 + 0.3 * rnd(d)) if norm != "l2" else (None, None)
    f = B.rope_frequencies(n, device="cuda")[0] if n else None
    pos = torch.randint(0, 100000, (Bn, T), generator=r, device="cuda", dtype=torch.int32)
    angle = pos.double()[..., None] * (f.double() if n else torch.zeros(0, dtype=torch.float64, device="cuda"))
    kw = dict(norm=norm, eps=1e-6, inv_freq=f, positions=pos, layout=layout, amplitude=1.25)
    yq, yk = B.qknorm_fwd(q, k, wq, wk, **kw)
    dq, dk = torch.full_like(dyq, float("nan")), torch.full_like(dyk, float("nan"))
    _, _, dwq, dwk = B.qknorm_bwd(q, k, dyq, dyk, wq, wk, dq=dq, dk=dk, **kw)
    torch.cuda.synchronize()
    half = 2.0 ** -8 if io == "bf16" else U
    for name, t, w, dy, y, dx, dw in (("q", q, wq, dyq, yq, dq, dwq), ("k", k, wk, dyk, yk, dk, dwk)):
        ry, rdx, rdw = reference(t, w, dy, angle, norm, 1e-6, 1.25, layout)
        close(y, ry, half, f"{what} y{name}")
        close(dx, rdx, half, f"{what} d{name}")
        close(dw, rdw, U, f"{what} dw{name}")


def test_gradients_past_32_bit_offsets():
    """2^20 + 3 tokens of 17 heads of 256 channels, 4.6e9 values: rows near the ends and in the
    middle against a call on these tokens alone, the weights' gradients against float64."""
    T, H, d, step = (1 << 20) + 3, 17, 256, 1 << 16
    r = torch.Generator(device="cuda").manual_seed(9)

    def fill():
        x = torch.empty((1, T, H, d), dtype=torch.bfloat16, device="cuda")
        for t in range(0, T, 1 << 18):
            n = min(T - t, 1 << 18)
            x[0, t:t + n] = torch.randn((n, H, d), generator=r, device="cuda")
        return x[:, :, :16].transpose(1, 2), x[:, :, 16:].transpose(1, 2)

    (q, k), (dyq, dyk) = fill(), fill()
    out = torch.full((1, T, H, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    w = 1 + 0.3 * torch.randn(d, generator=r, device="cuda")
    f = B.rope_frequencies(64, device="cuda")[0]
    kw = dict(norm="rms", inv_freq=f, layout="pairs")
    dq, dk, dwq, dwk = B.qknorm_bwd(q, k, dyq, dyk, w, w, dq=out[:, :, :16].transpose(1, 2),
                                    dk=out[:, :, 16:].transpose(1, 2), **kw)
    torch.cuda.synchronize()
    for t in (0, 12345, T // 2, T - 64):
        pos = torch.arange(t, t + 64, dtype=torch.int32, device="cuda")[None]
        n = slice(t, t + 64)
        one = B.qknorm_bwd(q[:, :, n], k[:, :, n], dyq[:, :, n], dyk[:, :, n], w, w, positions=pos, **kw)
        assert torch.equal(dq[:, :, n], one[0]) and torch.equal(dk[:, :, n], one[1]), t
    assert not bool(out.isnan().any())
    for x, dy, dw in ((q, dyq, dwq), (k, dyk, dwk)):
        ref, tol = torch.zeros(d, dtype=torch.float64, device="cuda"), torch.zeros(d, dtype=torch.float64, device="cuda")
        for t in range(0, T, step):
            n = slice(t, min(T, t + step))
            angle = torch.arange(t, n.stop, device="cuda", dtype=torch.float64)[None, :, None] * f.double()
            _, _, (a, b) = reference(x[:, :, n], w, dy[:, :, n], angle, "rms", 1e-6, 1.0, "pairs")
            ref, tol = ref + a, tol + b
        # each part's bound holds (d / 2 + 48 + 8 sqrt(its rows)); all rows': 8 sqrt(all of them)
        tol = tol * math.sqrt(T / step)
        close(dw, (ref, tol), U, "weights' gradients of 2^20 tokens")
