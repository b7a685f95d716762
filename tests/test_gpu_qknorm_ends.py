"""Rows of queries and keys at the ends of what qknorm_fwd and qknorm_bwd take: magnitudes far
from one, infinities and NaN where the definition copies a channel.  References and bounds
as in test_gpu_qknorm.py."""
import pytest
import torch

from tests.test_gpu_qknorm import close, make, reference
from xlstm_mlstm_matrix_amd import binding as B

pytestmark = pytest.mark.gpu


def cu(c):
    return {n: None if t is None else t.cuda() for n, t in c.items()}


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("shift,eps", [(50, 1e-6), (56, 0.0), (-30, 0.0), (-44, 0.0)])
@pytest.mark.parametrize("shape,n", [((2, 7, 3, 2, 64), 16), ((1, 9, 2, 1, 33), 5)], ids=str)
def test_rows_of_any_magnitude(io, norm, shift, eps, shape, n):
    """Rows of 2^shift: their squares, and one over them, are ordinary float32 numbers, the
    third power of one over their norm is not."""
    c = make(io, *shape, n, norm, 100, seed=shift)
    c["q"], c["k"] = c["q"] * 2.0 ** shift, c["k"] * 2.0 ** shift
    y, dx, dw = reference(c, norm, eps, "half", 1.25)
    g = cu(c)
    kw = dict(norm=norm, eps=eps, inv_freq=g["f"], positions=g["pos"], amplitude=1.25)
    got = B.qknorm_fwd(g["q"], g["k"], g["wq"], g["wk"], **kw) \
        + B.qknorm_bwd(g["q"], g["k"], g["dyq"], g["dyk"], g["wq"], g["wk"], **kw)
    torch.cuda.synchronize()
    for name, x, (ref, tol) in zip(("yq", "yk", "dq", "dk", "dwq", "dwk"), got, y + dx + dw):
        close(x, ref, tol, "f32" if name[:2] == "dw" else io, f"{io} {norm} 2^{shift} {name}")


def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("d,n", [(64, 16), (64, 0), (40, 3), (33, 8), (512, 8)])
def test_channels_that_are_not_rotated_are_copied(io, layout, d, n):
    """Without a norm and weights a channel behind the rotated ones is the input's, bit for
    bit, whatever its neighbours hold, and so is its gradient."""
    c = make(io, 2, 11, 3, 2, d, n, "none", 50, seed=d + n, weight=False)
    odd = (float("inf"), -float("inf"), float("nan"), -0.0, 3e38)
    g = cu(c)
    plain = {}
    for name in ("q", "k", "dyq", "dyk"):
        x = g[name].clone()
        plain[name] = x.clone()
        for i, value in enumerate(odd * 3):
            x[i % 2, i % x.shape[1], i % 11, 2 * n + (5 * i) % (d - 2 * n)] = value
        g[name] = x
    kw = dict(norm="none", inv_freq=g["f"], positions=g["pos"], layout=layout)
    got = B.qknorm_fwd(g["q"], g["k"], **kw) + B.qknorm_bwd(g["q"], g["k"], g["dyq"], g["dyk"], weight_grad=False, **kw)[:2]
    ref = B.qknorm_fwd(plain["q"], plain["k"], **kw) \
        + B.qknorm_bwd(plain["q"], plain["k"], plain["dyq"], plain["dyk"], weight_grad=False, **kw)[:2]
    torch.cuda.synchronize()
    for name, x, r in zip(("q", "k", "dyq", "dyk"), got, ref):
        a, b = x[..., 2 * n:], g[name][..., 2 * n:]
        same = (bits(a) == bits(b)) | (a.isnan() & b.isnan()).contiguous()
        assert bool(same.all()), (name, int((~same).sum()))
        assert torch.equal(x[..., :2 * n], r[..., :2 * n]), name
