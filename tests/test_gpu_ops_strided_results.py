"""Results of the gated delta rule and of the norm and rotation written into views of wider rows:
the values of a dense call, and not a bit changed around them."""
import pytest
import torch

from tests.test_gpu_deltarule import cu, ints, make
from xlstm_mlstm_matrix_amd import binding as B

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
MARK = -12345.0


class Around:
    """Buffers full of one value with a view for a result in the middle of each."""

    def __init__(self):
        self.held = []

    def rows(self, shape, dtype, pad, after=0):
        """[B, H, T, d] as token-major rows of d + pad + after elements, a token and a sequence to spare
        at both ends."""
        Bn, H, T, d = shape
        buf = torch.full((Bn + 2, T + 2, H, d + pad + after), MARK, dtype=dtype, device="cuda")
        view = buf[1:-1, 1:-1, :, pad:pad + d].permute(0, 2, 1, 3)
        self.held.append((buf, view))
        return view

    def gates(self, shape):
        buf = torch.full((shape[0] + 2, shape[2] + 2, 2 * shape[1] + 1), MARK, device="cuda")
        view = buf[1:-1, 1:-1, 1::2].transpose(1, 2)
        self.held.append((buf, view))
        return view

    def check(self, what):
        for i, (buf, view) in enumerate(self.held):
            view.fill_(MARK)
            assert bool((buf == torch.full((), MARK, dtype=buf.dtype, device="cuda")).all()), (what, i)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(3, 1, 2, 75, 48, 80), (2, 2, 2, 33, 128, 16), (1, 1, 1, 600, 16, 48),
                                   (16, 8, 16, 40, 80, 112), (8, 8, 8, 35, 240, 496)], ids=str)
def test_deltarule(io, shape):
    Bn, Hk, H, T, dk, dv = shape
    g = cu(make(io, *shape, seed=51))
    ln = ints([T, T // 3, 0][:Bn] + [T - 1] * max(Bn - 3, 0))
    a = [g[x] for x in ("q", "k", "v", "g", "beta")]
    dense = B.deltarule_fwd(*a, g["S0"], lengths=ln, scale=0.3) + B.deltarule_bwd(*a, g["do"], g["S0"], g["dS"], lengths=ln, scale=0.3)
    r, dt = Around(), DT[io]
    o = r.rows((Bn, H, T, dv), dt, 16, 8)
    kw = dict(dq=r.rows((Bn, Hk, T, dk), dt, 8, 8), dk=r.rows((Bn, Hk, T, dk), dt, 32), dv=r.rows((Bn, H, T, dv), dt, 8),
              dlog_decay=r.gates((Bn, H, T)), dbeta=r.gates((Bn, H, T)))
    got = B.deltarule_fwd(*a, g["S0"], lengths=ln, scale=0.3, o=o) \
        + B.deltarule_bwd(*a, g["do"], g["S0"], g["dS"], lengths=ln, scale=0.3, **kw)
    torch.cuda.synchronize()
    for i, (x, y) in enumerate(zip(got, dense)):
        assert torch.equal(x, y), i
    r.check(shape)
    r = Around()
    one = [x[:, :, 0] for x in a]
    ref, _ = B.deltarule_step(*one, g["S0"], scale=0.3, inplace=False)
    x, _ = B.deltarule_step(*one, g["S0"], scale=0.3, inplace=False, o=r.rows((Bn, H, 1, dv), dt, 16, 8)[:, :, 0])
    torch.cuda.synchronize()
    assert torch.equal(x, ref)
    r.check("step")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,n", [(64, 16), (128, 64), (33, 8), (1, 0), (96, 36), (512, 0), (511, 255)])
@pytest.mark.parametrize("pad", [8, 3])
def test_qknorm(io, d, n, pad):
    Bn, H, Hk, T = 2, 5, 3, 41
    gen = torch.Generator(device="cuda").manual_seed(d)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").to(DT[io])
    q, k, dyq, dyk = rnd(Bn, H, T, d), rnd(Bn, Hk, T, d), rnd(Bn, H, T, d), rnd(Bn, Hk, T, d)
    f = B.rope_frequencies(n, device="cuda")[0] if n else None
    for layout in ("half", "pairs"):
        kw = dict(inv_freq=f, layout=layout)
        # the same rows by single channels where the views' rows begin at odd places
        dense = B.qknorm_fwd(q, k, **kw) + B.qknorm_bwd(q, k, dyq, dyk, **kw)
        r = Around()
        view = lambda h: r.rows((Bn, h, T, d), DT[io], pad, pad)
        got = B.qknorm_fwd(q, k, yq=view(H), yk=view(Hk), **kw) \
            + B.qknorm_bwd(q, k, dyq, dyk, dq=view(H), dk=view(Hk), **kw)
        torch.cuda.synchronize()
        half = torch.finfo(DT[io]).eps
        for i, (x, y) in enumerate(zip(got, dense)):
            if pad == 8 and i < 4:
                assert torch.equal(x, y), (layout, i)
            else:
                # another grouping of the same sums: d of them in float32, 82 to 205 rows, one rounding
                size = float(y.float().abs().max())
                assert float((x.float() - y.float()).abs().max()) <= (half + (d + 256) * 2.0 ** -23) * size, (layout, i)
        r.check((d, n, layout))
