"""Seeded random-shape parity sweep of linear attention (forward, backward and
step) and of group norm (forward and backward) against float64.

Head sizes, tokens, lengths, decays (0 and 1 among them), states, strides, types,
activations and what a norm is taken over are drawn together from one seeded
generator.  Bounds are those of test_gpu_linattn_plans and test_gpu_groupnorm.
Every case prints its draw before it runs."""
import numpy as np
import pytest
import torch

from tests.test_gpu_groupnorm import run as norm_run
from tests.test_gpu_linattn import cu, make
from tests.test_gpu_linattn_plans import close, compare
from tests import linattn_dense as D
from xlstm_mlstm_matrix_amd import binding as B

pytestmark = pytest.mark.gpu


def draw_heads(r):
    log = lambda lo, hi: int(round(np.exp(r.uniform(np.log(lo), np.log(hi + 0.49)))))
    Bn, H = log(1, 6), log(1, 8)
    dk, dv = 16 * log(1, 16), 16 * log(1, 32)
    T = log(1, max(1, min(700, int(6e7 / (Bn * H * dk * dv) + 40))))
    decay = [float(r.choice([-float("inf"), 0.0, -1e-4, -2.0 ** -r.uniform(-3, 10)], p=[0.05, 0.1, 0.1, 0.75]))
             for _ in range(H)]
    return Bn, H, T, dk, dv, decay


def token_major(t):
    """The same [B, H, T, d] values as a view of wider token-major rows."""
    if t.dim() != 4:
        return t
    Bn, H, T, d = t.shape
    rows = torch.full((Bn, T, H, d + 16), float("nan"), dtype=t.dtype, device="cuda")
    view = rows[..., 16:].permute(0, 2, 1, 3)
    view.copy_(t)
    return view


@pytest.mark.parametrize("seed", range(40))
def test_linattn(seed):
    r = np.random.default_rng(8100 + seed)
    io = ("f32", "bf16")[int(r.integers(2))]
    Bn, H, T, dk, dv, decay = draw_heads(r)
    lengths = [int(x) for x in r.integers(-1, T + 3, Bn)] if r.random() < 0.5 else None
    state, strided = bool(r.integers(2)), bool(r.integers(2))
    what = f"{io} B{Bn} H{H} T{T} dk{dk} dv{dv} lengths {lengths} state {state} strided {strided} decay {decay}"
    d = make(io, Bn, H, T, dk, dv, seed=seed, state=state, decay=decay)
    g = cu(d)
    if strided:
        g = {n: token_major(t) if n in ("q", "k", "v", "do") else t for n, t in g.items()}
    compare(d, io, lengths, dk ** -0.5, what, g)


@pytest.mark.parametrize("seed", range(16))
def test_linattn_step(seed):
    r = np.random.default_rng(8300 + seed)
    io = ("f32", "bf16")[int(r.integers(2))]
    Bn, H, _, dk, dv, decay = draw_heads(r)
    d = make(io, Bn, H, 1, dk, dv, seed=seed, state=bool(r.integers(2)), decay=decay)
    g = cu(d)
    what = f"{io} step B{Bn} H{H} dk{dk} dv{dv} state {d['S0'] is not None}"
    print(f"[linattn] {what}", flush=True)
    o, S = B.linattn_step(*(g[n][:, :, 0] for n in "qkv"), g["g"], g["S0"], scale=0.4, inplace=False)
    (ro, rS), _ = D.both(d, scale=0.4)
    (Ao, AS), _ = D.both(d, scale=0.4, magnitudes=True)
    close(o[:, :, None], ro, Ao, io, dk, what + " o")
    close(S, rS, AS, "f32", 0, what + " S")


@pytest.mark.parametrize("seed", range(32))
def test_groupnorm(seed):
    r = np.random.default_rng(8500 + seed)
    log = lambda lo, hi: int(round(np.exp(r.uniform(np.log(lo), np.log(hi + 0.49)))))
    over = ("token", "sequence")[int(r.integers(2))]
    N, G, D_ = log(1, 8), log(1, 40), log(1, 3000 if over == "token" else 300)
    S = log(1, max(1, min(4000, int(2e6 / (N * G * D_)))))
    norm_run(("f32", "bf16")[int(r.integers(2))], (N, S, G, D_), over, ("none", "silu", "gelu")[int(r.integers(3))],
             head_major=bool(r.integers(2)), seed=seed, mean=float(r.choice([0.0, 0.5, -20.0])),
             affine=bool(r.random() < 0.8))
