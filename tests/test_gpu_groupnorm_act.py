"""The activations of group norm over their whole range, float32: with weights of
zero the result is act(bias), and the bias's gradient under dy = 1 its derivative.

u = 2^-24.  GELU z Phi(z): for z < 0, Phi is a polynomial (6 u) in a quotient (3 u)
times a power whose exponent z^2 / 2 is rounded three times (1.3 z^2 u) and which is
good to 2 u itself; five products and roundings more: (16 + 1.3 z^2) u of itself.  For
z >= 0 it is 1 minus that.  Its derivative Phi + z phi(z) has the same errors in each
term.  SiLU z s(z), s = 1 / (1 + e^-z): the power is off by (1.5 |z| + 2) u, the rest
adds 4 u; its derivative s (1 + z (1 - s)) has s twice.
"""
import math

import pytest
import torch

from xlstm_mlstm_matrix_amd import binding as B

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("over", ["token", "sequence"])
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_activation_and_derivative(act, over):
    z = torch.cat([torch.linspace(-12, 12, 4000), torch.logspace(-6, 0, 48), -torch.logspace(-6, 0, 48)]).cuda()
    bias = z.reshape(8, 512)
    x = torch.randn((1, 1, 8, 512), generator=torch.Generator(device="cuda").manual_seed(0), device="cuda")
    w = torch.zeros_like(bias)
    y, m, r = B.groupnorm_fwd(x, w, bias, act=act, over=over)
    _, _, db = B.groupnorm_bwd(x, torch.ones_like(x), m, r, w, bias, act=act, over=over)
    zd = bias.double()
    if act == "gelu":
        # the tails from erfc, whose relative precision holds there
        P = 0.5 * torch.special.erfc(-zd / math.sqrt(2.0))
        d = torch.exp(-zd * zd / 2) / math.sqrt(2 * math.pi)
        c = torch.where(zd < 0, 16 + 1.3 * zd * zd, torch.full_like(zd, 12))
        ref, tol = zd * P, c * U * (zd * P).abs()
        dref, dtol = P + zd * d, c * U * P + (8 + 1.3 * zd * zd) * U * (zd * d).abs()
    else:
        s = torch.sigmoid(zd)
        c = 1.5 * zd.abs() * (1 - s) + 8     # the power's error reaches s by 1 - s
        ref, tol = zd * s, c * U * (zd * s).abs()
        dref = s * (1 + zd * (1 - s))
        dtol = U * s * (c * (1 + (zd * (1 - s)).abs()) + (1.5 * zd.abs() + 8) * zd.abs() * s)
    for what, a, b, t in (("value", y[0, 0], ref, tol), ("derivative", db, dref, dtol)):
        bad = ((a.double() - b).abs() / (t + 1e-37)).max().item()
        print(f"[groupnorm] {act} {over} {what}: {bad:.3f} of the bound", flush=True)
        assert bad <= 1.0, (what, bad)
