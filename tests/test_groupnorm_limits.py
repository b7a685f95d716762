"""Group norm at the sizes where a launch would have 2^32 threads or more: the
calls go in several launches.  Float64 on the device.

Bounds as in test_gpu_groupnorm, for groups of at most 4 values between 1 and 2
in magnitude, one up and one down in turn, so that rstd is at most 1 and |xh| at
most 2: the mean is off by e = 65 u mean|x| (u = 2^-24), xh by rstd (e + u |x|) +
65 u |xh| + (e rstd)^2 |xh| < 2e-5.  y is one product of that by a weight below
1.5, dx three by factors below 2: 2e-4 leaves what rounding them adds.
"""
import pytest
import torch

from xlstm_mlstm_matrix_amd import binding as B

OK, SHAPE = 0, 2


def data(N, S, G, D, dt):
    """Values of magnitude 1 to 2, one up and one down in turn."""
    r = torch.Generator(device="cuda").manual_seed(8)
    x = torch.rand((N, S, G, D), generator=r, device="cuda") + 1.0
    x[..., 1::2] *= -1
    w = torch.rand((G, D), generator=r, device="cuda") + 0.5
    return x.to(dt), torch.rand((N, S, G, D), generator=r, device="cuda").to(dt), w, w - 1.0


def reference(x, dy, w, b, dims, part):
    """(y, dx) of samples or groups `part`, and their dz and dz * xh, in float64."""
    n, g = part
    x, dy, w, b = x[n][:, :, g].double(), dy[n][:, :, g].double(), w[g].double(), b[g].double()
    m = x.mean(dims, keepdim=True)
    r = (((x - m) ** 2).mean(dims, keepdim=True) + 1e-5).rsqrt()
    xh = (x - m) * r
    u = dy * w
    dx = r * (u - u.mean(dims, keepdim=True) - xh * (u * xh).mean(dims, keepdim=True))
    return xh * w + b, dx, dy, dy * xh


def check(x, ref, half, what):
    bad = ((x.double() - ref).abs() / (half * 1.01 * ref.abs() + 2e-4)).max().item()
    print(f"[groupnorm] {what}: {bad:.3f} of the bound", flush=True)
    assert bad <= 1.0, (what, bad)


@pytest.mark.gpu
@pytest.mark.parametrize("N,G", [((1 << 24) + 5, 1), (1 << 17, 32 + 1)], ids=str)
def test_backward_of_many_samples_and_groups(N, G):
    """2^22 groups and more in the combining launch of 1024 threads each; the
    first case has 2^24 workgroups in the others too."""
    x, dy, w, b = data(N, 1, G, 2, torch.bfloat16)
    y, m, r = B.groupnorm_fwd(x, w, b, over="sequence")
    dx, dw, db = B.groupnorm_bwd(x, dy, m, r, w, b, over="sequence")
    torch.cuda.synchronize()
    sdz = sdx = 0
    for n in torch.arange(N, device="cuda").split(1 << 22):
        ry, rdx, dz, dzx = reference(x, dy, w, b, (1, 3), (slice(int(n[0]), int(n[-1]) + 1), slice(None)))
        part = slice(int(n[0]), int(n[-1]) + 1)
        check(y[part], ry, 2.0 ** -8, "y")
        check(dx[part], rdx, 2.0 ** -8, "dx")
        sdz, sdx = sdz + dz.sum((0, 1)), sdx + dzx.sum((0, 1))
    # terms of one sign; 64 threads add every 64th sample's, then a tree
    k = (N / 64 + 64) * 2.0 ** -24
    assert bool(((db.double() - sdz).abs() <= k * sdz.abs()).all())
    assert bool(((dw.double() - sdx).abs() <= (k + 2e-4) * sdx.abs()).all())


@pytest.mark.gpu
def test_forward_of_many_groups():
    """2^26 groups of a workgroup of 64 threads each."""
    N = (1 << 26) + 3
    x, _, w, b = data(N, 1, 1, 2, torch.bfloat16)
    y = B.groupnorm_fwd(x, w, b, over="sequence", return_stats=False)
    torch.cuda.synchronize()
    for n in range(0, N, 1 << 24):
        ry, *_ = reference(x, x, w, b, (1, 3), (slice(n, n + (1 << 24)), slice(None)))
        check(y[n:n + (1 << 24)], ry, 2.0 ** -8, "y")


@pytest.mark.gpu
def test_many_groups_over_tokens():
    """2^24 groups of one position (a workgroup each) and 2^26 weights, whose
    gradients are summed by 1024 threads for 16 of them."""
    G = (1 << 24) + 1
    x, dy, w, b = data(1, 1, G, 4, torch.float32)
    y, m, r = B.groupnorm_fwd(x, w, b)
    dx, dw, db = B.groupnorm_bwd(x, dy, m, r, w, b)
    torch.cuda.synchronize()
    for g in range(0, G, 1 << 22):
        part = slice(g, g + (1 << 22))
        ry, rdx, dz, dzx = reference(x, dy, w, b, (3,), (slice(None), part))
        check(y[:, :, part], ry, 2.0 ** -24, "y")
        check(dx[:, :, part], rdx, 2.0 ** -24, "dx")
        assert torch.equal(db[part].double(), dz[0, 0])
        check(dw[part], dzx[0, 0], 2.0 ** -24, "dw")


def test_sizes_past_the_limits_are_refused():
    """N S, G D, N G below 2^30, N ceil(G D / 64) below 2^28, checked without a device."""
    import ctypes
    n = ctypes.c_size_t(0)
    q = lambda *a: B.lib().mlstm_groupnorm_workspace_size(*a, 1, 1, 1, ctypes.byref(n))
    assert q(1 << 30, 1, 1, 1) == SHAPE and q(1, 1, 1 << 15, 1 << 15) == SHAPE
    assert q(1 << 28, 1, 1, 64) == SHAPE and q((1 << 28) - 1, 1, 1, 64) == OK
    assert q(1 << 15, 1, 1 << 15, 1) == SHAPE and q(1 << 15, 1, 1 << 14, 1) == OK
    assert q(1, (1 << 30) - 1, 1, 1) == OK
