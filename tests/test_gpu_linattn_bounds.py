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


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_state_through_many_segments(io):
    """A state that decays slowly through 512 segments is not pulled one way.

    Each segment rounds an element twice, by at most u of it either way: over 511
    segments a standard deviation below sqrt(2 * 511 / 3) u = 19 u, in the mean of
    4096 elements 0.3 u.  What all elements share: the decay's logarithm in base 2
    (|g| T u <= 1.1 u), the last segment's power (4 u) and the tokens' own weights
    (40 u of at most a tenth of the state): 10 u.  So the mean is held to 12 u; a
    rounded factor may add 511 u / 2.
    """
    T, d = 65536, 64
    r = np.random.default_rng(17)
    # decays whose power of a 128-token segment lies far from a float
    cand = -r.uniform(2e-6, 1.6e-5, 4000).astype(np.float32)
    f = np.exp2((cand * np.float32(1.4426950408889634)).astype(np.float64) * 128)
    off = (f.astype(np.float32) - f) / U
    for g in cand[[int(off.argmin()), int(off.argmax())]]:
        k, v = (torch.from_numpy(r.normal(0, s, (1, 1, T, d)).astype(np.float32)) for s in (0.01, 1.0))
        k, v = ((x.bfloat16() if io == "bf16" else x).cuda() for x in (k, v))
        S0 = torch.from_numpy(r.uniform(100, 200, (1, 1, d, d)).astype(np.float32)).cuda()
        decay = torch.tensor([g], device="cuda")
        _, S = B.linattn_fwd(k, k, v, decay, S0)
        w = torch.exp(decay.double() * torch.arange(T - 1, -1, -1, device="cuda"))[:, None]
        ref = S0.double() * torch.exp(decay.double() * T) + (k[0, 0].double() * w).T @ v[0, 0].double()
        e = (S.double() / ref - 1).mean().item() / U
        print(f"[linattn] {io} decay {g:.3e}: mean error {e:.2f} u", flush=True)
        assert abs(e) <= 12


@pytest.mark.parametrize("T", [1, 5, 32, 40])
def test_states_of_short_bfloat16_sequences(T):
    """A state that is handed out is as float32 sums leave it: u for each sum and
    40 u for a product's weight, a product of five powers each good to 2 u and
    rounded four times, of exponents below 3.  Two parts of it instead of three
    would be off by up to 2^-16 = 256 u.
    """
    d = make("bf16", 2, 3, T, 64, 64, seed=T, decay=[-0.05, -0.01, 0.0])
    g, m = cu(d), mag(d)
    _, S = B.linattn_fwd(g["q"], g["k"], g["v"], g["g"], g["S0"])
    _, ref = O.linattn_forward(d["q"], d["k"], d["v"], d["g"], d["S0"])
    _, A = O.linattn_forward(m["q"], m["k"], m["v"], m["g"], m["S0"])
    bad = (np.abs(S.double().cpu().numpy() - ref) / ((40 + T) * U * A)).max()
    print(f"[linattn] state of {T} tokens: {bad:.3f} of the bound", flush=True)
    assert bad <= 1.0
