"""GPU parity of linear attention in every split of the work that its plan can
choose: rows padded to 64, 128, 256 and 512, blocks of 64 and 128 columns, one or
several of them, whole sequences and segments, forward and backward.

The float64 reference is the unrolled form.  Bounds: u = 2^-24, A the operator
applied to magnitudes, N the terms of a sum.  float32: (N + 64) u A.  bfloat16
outputs: 2^-8 of the value for its rounding, 2^-16 A for each of up to three
operands that are carried in two parts, and the float32 term; states 2^-16 A and
the float32 term.
"""
import numpy as np
import pytest
import torch

from tests import linattn_dense as D
from tests.test_gpu_linattn import cu, make
from xlstm_mlstm_matrix_amd import binding as B

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def close(x, ref, A, io, N, what, state=False):
    x = x.detach().double().cpu().numpy()
    assert x.shape == ref.shape and np.all(np.isfinite(x)), what
    tol = (N + 64) * U * A
    if io == "bf16":
        tol = tol + 2.0 ** -16 * A if state else 1.01 * (tol + 2.0 ** -8 * np.abs(ref) + 3 * 2.0 ** -16 * A)
    bad = (np.abs(x - ref) / (tol + 1e-30)).max()
    print(f"[linattn] {what}: {bad:.3f} of the bound", flush=True)
    assert bad <= 1.0, (what, float(bad))


def compare(d, io, lengths=None, scale=1.0, what="", g=None):
    """Forward and backward, with the state handed out and without."""
    g = cu(d) if g is None else g
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    print(f"[linattn] {what}", flush=True)
    o, S = B.linattn_fwd(g["q"], g["k"], g["v"], g["g"], g["S0"], lengths=ln, scale=scale)
    o2 = B.linattn_fwd(g["q"], g["k"], g["v"], g["g"], g["S0"], lengths=ln, scale=scale, return_state=False)
    gr = B.linattn_bwd(g["q"], g["k"], g["v"], g["g"], g["do"], g["S0"], g["dS"], lengths=ln, scale=scale,
                       state_grad=True)
    gr2 = B.linattn_bwd(g["q"], g["k"], g["v"], g["g"], g["do"], g["S0"], g["dS"], lengths=ln, scale=scale)
    torch.cuda.synchronize()
    (ro, rS), rg = D.both(d, lengths, scale)
    (Ao, AS), Ag = D.both(d, lengths, scale, magnitudes=True)
    N = d["q"].shape[2] + 2 * max(d["q"].shape[3], d["v"].shape[3])
    close(o, ro, Ao, io, N, what + " o")
    close(o2, ro, Ao, io, N, what + " o, no state")
    close(S, rS, AS, io, N, what + " S", state=True)
    for n, x, r, a in zip(("dq", "dk", "dv", "dS0"), gr, rg, Ag):
        close(x, r, a, io, N, f"{what} {n}", state=n == "dS0")
    for n, x, r, a in zip(("dq", "dk", "dv"), gr2, rg, Ag):
        close(x, r, a, io, N, f"{what} {n}, no state")


# B, H, T, dk, dv; lengths
SHAPES = [((1, 2, 520, 256, 512), None), ((2, 1, 300, 256, 512), [300, 71]), ((1, 1, 700, 240, 272), None),
          ((1, 1, 400, 256, 64), None), ((1, 2, 40, 112, 512), None), ((4, 16, 33, 48, 128), None),
          ((1, 2, 300, 112, 208), None), ((1, 2, 400, 128, 128), None), ((3, 1, 600, 64, 400), [600, 0, 130]),
          ((8, 16, 40, 64, 128), [40, 39, 33, 32, 31, 1, 0, 40]), ((4, 8, 40, 256, 512), None),
          ((4, 16, 70, 128, 128), None), ((1, 2, 300, 112, 400), None), ((16, 16, 33, 128, 256), None)]


@pytest.mark.parametrize("shape,lengths", SHAPES, ids=str)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_every_split(io, shape, lengths):
    compare(make(io, *shape, seed=sum(shape)), io, lengths, shape[3] ** -0.5, f"{io} {shape}")
