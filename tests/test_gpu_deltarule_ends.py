"""Calls of the gated delta rule whose own values are not finite: what the header says of the
rows behind a sequence holds all the same, and so does how far a NaN or an infinity reaches."""
import pytest
import torch

from tests.test_gpu_deltarule import cu, ints, make
from xlstm_mlstm_matrix_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("heads", [(2, 2), (1, 2)], ids=["own", "shared"])
@pytest.mark.parametrize("dk,dv", [(64, 80), (128, 64), (240, 48)])
@pytest.mark.parametrize("name", ["q", "k", "v", "do", "g", "beta", "S0", "dS"])
def test_rows_behind_a_sequence_of_nan_are_zeros(io, heads, dk, dv, name):
    """A NaN in a sequence's own tokens or its states reaches no row behind its length and no other
    sequence."""
    T, lengths = 100, [100, 70, 33, 5]
    d = make(io, 4, *heads, T, dk, dv, seed=31)
    g = cu(d)
    def run():
        a = [g[x] for x in ("q", "k", "v", "g", "beta")]
        o, S = B.deltarule_fwd(*a, g["S0"], lengths=ints(lengths), scale=0.2)
        return (o, S) + B.deltarule_bwd(*a, g["do"], g["S0"], g["dS"], lengths=ints(lengths), scale=0.2, state_grad=True)
    clean = run()
    for b in (1, 2, 3):
        if name in ("S0", "dS"):
            g[name][b, :, 3, 5] = float("nan")
        else:
            g[name][b, :, lengths[b] // 2] = float("nan")
    got = run()
    torch.cuda.synchronize()
    for i, (x, y) in enumerate(zip(got, clean)):
        assert torch.equal(x[0], y[0]), i
    for i in (0, 2, 3, 4, 5, 6):       # o, dq, dk, dv, dg, dbeta
        for b, n in enumerate(lengths):
            assert bool((got[i][b, :, n:] == 0).all()), (i, b)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 2, 4, 150, 48, 80), (2, 1, 2, 700, 64, 64), (1, 2, 2, 600, 240, 32),
                                   (16, 8, 16, 100, 64, 128), (8, 8, 8, 70, 256, 496)], ids=str)
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_values_that_are_not_finite_stay_in_their_head(io, shape, value):
    """In one head of the last sequence (of 64 columns a workgroup, of 128, of segments): no other
    head and no earlier chunk of its own changes a bit."""
    Bn, Hk, H, T, dk, dv = shape
    per = H // Hk
    d = make(io, *shape, seed=33)
    clean = cu(d)

    def run(g):
        a = [g[x] for x in ("q", "k", "v", "g", "beta")]
        out = B.deltarule_fwd(*a, g["S0"], scale=0.2)
        return out + B.deltarule_bwd(*a, g["do"], g["S0"], g["dS"], scale=0.2, state_grad=True)

    ref = run(clean)
    at = T // 2
    for name in ("q", "k", "v", "do", "beta", "S0", "dS") + (() if value > 0 else ("g",)):
        g = {n: x.clone() for n, x in clean.items()}
        hk = Hk - 1
        if name in ("S0", "dS"):
            g[name][-1, hk * per, 3, 5] = value
        else:
            g[name][-1, hk if name in ("q", "k") else hk * per, at] = value
        got = run(g)
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(got, ref)):
            heads = x.shape[1]
            bad = [hk] if heads == Hk and heads != H else [hk * per + j for j in range(per if name in ("q", "k") else 1)]
            keep = torch.ones(Bn, heads, dtype=torch.bool, device="cuda")
            keep[-1, bad] = False
            assert torch.equal(x[keep], y[keep]), (name, i)
            if i == 0 and name not in ("S0", "dS", "do"):
                first = at // 32 * 32
                assert torch.equal(x[:, :, :first], y[:, :, :first]), name
            if i == 0 and name in ("dS", "do"):
                assert torch.equal(x, y), name
