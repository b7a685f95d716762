"""Tighter bounds on linear attention than parity asks for: bfloat16 outputs are
float32 work rounded once.

With A the operator applied to the magnitudes of all inputs and N the terms of a
sum, an output is off by 2^-8 |o| for its own rounding, by 2^-16 A for each
operand that is carried in two bfloat16 parts (the read-out's copy of the state,
the scores, and, where no state is handed out, what each token adds to the
state), and by (N + 64) 2^-24 A for float32 products, decays and sums.  1.01
covers what one of these does to another.
"""
import numpy as np
import pytest
import torch

from oracle import ops as O
from tests.test_gpu_linattn import cu, mag, make
from xlstm_mlstm_matrix_amd import binding as B

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def close(x, ref, A, N, parts, what):
    x = x.detach().double().cpu().numpy()
    tol = 1.01 * (2.0 ** -8 * np.abs(ref) + (parts * 2.0 ** -16 + (N + 64) * U) * A) + 1e-30
    bad = (np.abs(x - ref) / tol).max()
    print(f"[linattn] {what}: {bad:.3f} of the bound", flush=True)
    assert bad <= 1.0, (what, float(bad))


@pytest.mark.parametrize("shape", [(2, 2, 5, 16, 48), (1, 3, 1, 64, 64), (2, 2, 150, 64, 64), (1, 2, 200, 128, 128),
                                   (1, 2, 700, 64, 128), (1, 1, 120, 256, 512)], ids=str)
@pytest.mark.parametrize("state", [True, False])
def test_bfloat16_outputs_are_rounded_once(shape, state):
    """A single rounded copy of the state, or a single rounded score, is off by
    2^-8 of the terms it multiplies: where they cancel, far past this bound."""
    d = make("bf16", *shape, seed=21, state=True)
    g, m = cu(d), mag(d)
    s, N = shape[3] ** -0.5, shape[2] + 2 * max(shape[3:])
    what = f"{shape} state {state}"
    print(f"[linattn] {what}", flush=True)
    o = B.linattn_fwd(g["q"], g["k"], g["v"], g["g"], g["S0"], scale=s, return_state=state)
    gr = B.linattn_bwd(g["q"], g["k"], g["v"], g["g"], g["do"], g["S0"], g["dS"], scale=s, state_grad=state)
    torch.cuda.synchronize()
    fw = lambda x: O.linattn_forward(x["q"], x["k"], x["v"], x["g"], x["S0"], scale=s)[0]
    bw = lambda x: O.linattn_backward(x["q"], x["k"], x["v"], x["g"], x["do"], x["S0"], x["dS"], scale=s)
    close(o[0] if state else o, fw(d), fw(m), N, 2 if state else 3, what + " o")
    for n, x, r, a in zip(("dq", "dk", "dv"), gr, bw(d), bw(m)):
        # only the passes that share a launch with the state's carry it in three parts
        close(x, r, a, N, 3, f"{what} {n}")
