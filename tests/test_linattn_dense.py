"""The unrolled form of linear attention against the recurrence of the oracle."""
import numpy as np
import pytest
import torch

from oracle import ops as O
from tests import linattn_dense as D


@pytest.mark.parametrize("lengths", [None, [9, 0, 4]])
@pytest.mark.parametrize("state", [True, False])
def test_unrolled_equals_recurrent(lengths, state):
    r = np.random.default_rng(2)
    t = lambda *s: torch.from_numpy(r.normal(size=s))
    d = {"q": t(3, 4, 9, 5), "k": t(3, 4, 9, 5), "v": t(3, 4, 9, 3), "do": t(3, 4, 9, 3),
         "g": torch.tensor([-float("inf"), -0.7, -0.01, 0.0], dtype=torch.float64),
         "S0": t(3, 4, 5, 3) if state else None, "dS": t(3, 4, 5, 3) if state else None}
    out, grad = D.both(d, lengths, 0.6)
    ref = O.linattn_forward(d["q"], d["k"], d["v"], d["g"], d["S0"], lengths, 0.6)
    gref = O.linattn_backward(d["q"], d["k"], d["v"], d["g"], d["do"], d["S0"], d["dS"], lengths, 0.6)
    for a, b in zip(out + grad, ref + gref):
        np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-12)
