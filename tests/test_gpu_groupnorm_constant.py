"""Constant groups of group norm, and means far from zero.

A constant group's x - mean is exactly 0, so the result is exactly the bias and the
saved mean exactly the value, for values whose sums over a group are not floats.
The variance is what rounding leaves of it: a mean's first step is off by a few u
of the value c (u = 2^-24), and the square of that is taken away again up to a few
u of itself: (8 u c)^2 * 8 u, which is below 1e-5 of eps for c = 12345.678.
"""
import pytest
import torch

from xlstm_mlstm_matrix_amd import binding as B

pytestmark = pytest.mark.gpu

VALUES = [12345.678, 0.1, -3.3e-5, -777.7]


# groups in a few lanes, in a wavefront, in a workgroup's loop; in a workgroup's registers; in blocks of positions
CASES = [("token", 5, D) for D in (1, 7, 48, 96, 112, 250, 513, 2047, 5000)] \
    + [("sequence", 37, D) for D in (1, 10, 48, 112)] + [("sequence", 5, 3000)] \
    + [("sequence", 3001, D) for D in (7, 48, 112)] + [("sequence", 300, 100)]


@pytest.mark.parametrize("over,S,D", CASES, ids=str)
@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_constant_groups_give_their_bias(io, over, S, D):
    N, G = 2, len(VALUES)
    val = torch.tensor(VALUES, device="cuda").to(io)
    x = val[:, None].expand(N, S, G, D).contiguous()
    r = torch.Generator(device="cuda").manual_seed(D)
    w, b = (torch.randn((G, D), generator=r, device="cuda") for _ in range(2))
    print(f"[groupnorm] constant {io} {over} {S} x {D}", flush=True)
    y, m, rs = B.groupnorm_fwd(x, w, b, over=over)
    assert torch.equal(y, b.to(io).expand_as(y))
    assert torch.equal(m, val.float().expand_as(m))
    # half of that, and the root is good to 4 u
    assert bool(((rs.double() * 1e-5 ** 0.5 - 1).abs() <= 0.5e-5 + 4 * 2.0 ** -24).all())


FAR = [("token", 9, 96), ("token", 9, 750), ("token", 3, 5000), ("sequence", 64, 48), ("sequence", 1000, 48)]


@pytest.mark.parametrize("over,S,D", FAR, ids=str)
@pytest.mark.parametrize("outlier", [0.0, 1e5])
def test_means_to_their_last_bit(over, S, D, outlier):
    """Values of spread 1 around 3000, the first of each group an outlier or not.

    The mean's last step adds a correction to a value: u |mean| for that addition,
    and the correction, a mean of n distances d from a point a few u max|x| off the
    mean: (n / 64 + 64) u mean|d|, with each d rounded, u mean|d| more.
    """
    x = torch.randn((2, S, 3, D), generator=torch.Generator(device="cuda").manual_seed(D), device="cuda") + 3000.0
    if over == "token":
        x[..., 0] += outlier
    else:
        x[:, 0, :, 0] += outlier
    _, m, r = B.groupnorm_fwd(x, over=over)
    dims = (3,) if over == "token" else (1, 3)
    n, X = D * (1 if over == "token" else S), x.double()
    mu = X.mean(dims, keepdim=True)
    spread = (X - mu).abs().mean(dims)
    mu = mu.reshape(m.shape)
    bad = ((m.double() - mu).abs() / (2.0 ** -24 * (1.01 * mu.abs() + (n / 64 + 65) * spread))).max().item()
    print(f"[groupnorm] mean {over} {S} x {D} outlier {outlier}: {bad:.3f} of the bound", flush=True)
    assert bad <= 1.0
