"""Calls of the gated delta rule whose own values are not finite: what the header says of the
rows behind a sequence holds all the same."""
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
