"""The gated delta rule where there are heads enough for 128 columns a workgroup, which
smaller calls never take: forward and gradients against float64 (bounds as in
deltarule_bounds.py).

Some heads of a few sequences are repeated until a call is large enough; the copies have to
come out bit for bit alike, so that every workgroup's result is held to float64."""
import pytest
import torch

from tests import deltarule_bounds as D
from tests.test_gpu_deltarule import GRADS, cu, ints, make
from xlstm_mlstm_matrix_amd import binding as B

pytestmark = pytest.mark.gpu

WIDE = 256  # blocks of up to 128 columns in a call

# B, Hk, H, T, dk, dv: padded rows and columns, whole tiles, shared heads, a column block
# that is half empty or nearly so
SHAPES = [(2, 2, 4, 100, 48, 80), (1, 2, 2, 129, 64, 64), (2, 2, 2, 70, 64, 128), (2, 1, 2, 70, 112, 208),
          (1, 1, 2, 131, 128, 128), (2, 2, 2, 40, 96, 320), (1, 2, 2, 130, 240, 496), (2, 1, 2, 65, 256, 512),
          (2, 3, 3, 33, 16, 16)]


def repeated(d, lengths, shape):
    """The call's inputs, its sequences repeated until its plan is the wide one."""
    Bn, _, H, _, _, dv = shape
    n = -(-WIDE // (Bn * H * -(-dv // 128)))
    g = {k: None if x is None else x.repeat(n, *[1] * (x.dim() - 1)) for k, x in cu(d).items()}
    return g, ints(lengths * n if lengths else None), n


def alike(got, n, what):
    for i, x in enumerate(got):
        x = x.reshape(n, -1, *x.shape[1:])
        assert torch.equal(x, x[:1].expand_as(x)), (what, i)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_wide_walks(io, shape):
    Bn, T = shape[0], shape[3]
    lengths = [T, T - 35 if T > 35 else 7][:Bn] if Bn > 1 else None
    d = make(io, *shape, seed=40 + sum(shape))
    if lengths:
        for name in ("q", "k", "v", "do", "g", "beta"):
            d[name][1, :, lengths[1]:] = 0
    g, ln, n = repeated(d, lengths, shape)
    what = f"{io} wide {shape} x {n}"
    print(f"[delta] {what}", flush=True)
    a = [g[x] for x in ("q", "k", "v", "g", "beta")]
    s = shape[4] ** -0.5
    got = B.deltarule_fwd(*a, g["S0"], lengths=ln, scale=s) \
        + B.deltarule_bwd(*a, g["do"], g["S0"], g["dS"], lengths=ln, scale=s, state_grad=True)
    torch.cuda.synchronize()
    alike(got, n, what)
    w = D.sweep(d, lengths, s)
    D.check(w, dict(zip(("o", "S") + GRADS, (x[:Bn] for x in got))), io, what)


@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[4], SHAPES[6]], ids=str)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_wide_walks_without_a_state(io, shape):
    """No state given or asked for (fewer parts of it in bfloat16), and the final state written
    over the initial one."""
    Bn = shape[0]
    d = make(io, *shape, seed=60 + sum(shape))
    g, _, n = repeated(d, None, shape)
    what = f"{io} wide, no state {shape} x {n}"
    print(f"[delta] {what}", flush=True)
    a = [g[x] for x in ("q", "k", "v", "g", "beta")]
    s = shape[4] ** -0.5
    o = B.deltarule_fwd(*a, scale=s, return_state=False)
    back = B.deltarule_bwd(*a, g["do"], scale=s)
    o2, S = B.deltarule_fwd(*a, g["S0"], scale=s)
    state = g["S0"].clone()
    o3, S3 = B.deltarule_fwd(*a, state, scale=s, S_T=state)
    torch.cuda.synchronize()
    assert torch.equal(o2, o3) and torch.equal(S, S3)
    alike((o,) + back, n, what)
    D.check(D.sweep({**d, "S0": None, "dS": None}, None, s), dict(zip(("o",) + GRADS, (x[:Bn] for x in (o,) + back))), io, what)


def test_wide_is_the_narrow_walk():
    """The same heads in a call of 64 columns a workgroup: float32 results differ by sums' order
    within a product at the most, so by no more than the bound of both."""
    shape = (1, 2, 2, 96, 64, 128)
    d = make("f32", *shape, seed=77)
    g, _, n = repeated(d, None, shape)
    one = cu(d)
    call = lambda x: B.deltarule_fwd(*(x[k] for k in ("q", "k", "v", "g", "beta")), x["S0"], scale=0.125)
    w = D.sweep({**d, "do": None}, None, 0.125)
    for got in (call(g), call(one)):
        torch.cuda.synchronize()
        D.check(w, {"o": got[0][:1], "S": got[1][:1]}, "f32", f"wide against narrow x {got[0].shape[0]}")


# heads, d_qk, d_v: 64 columns a workgroup (exactly and with a remainder), 128 columns (the same), and
# past 320 MB
STEPS = [(512, 64, 64), (300, 80, 112), (1000, 16, 96), (512, 128, 128), (300, 48, 144), (520, 240, 208), (100, 256, 512),
         (300, 112, 272), (700, 256, 512), (5000, 128, 144), (12000, 16, 512)]


@pytest.mark.parametrize("heads,dk,dv", STEPS, ids=str)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_steps_of_many_heads(io, heads, dk, dv):
    """deltarule_step on states of the sizes that its kernels are chosen by: in place, from one
    tensor into another, from the zero state; float64 on the device.

    With u = beta (v - e^g S^T k): e^g is good to 8 U, a sum over d_qk to (d_qk + 16) U of its terms'
    magnitudes whatever its order, a handful of single roundings: the state to 16 U e^g |S| and
    (d_qk + 64) U |k| |u|, o = scale (e^g S^T q + (q . k) u) to (2 d_qk + 128) U of its terms, each
    taken with the magnitudes of everything in it, and bfloat16 to 2^-8 of itself more."""
    H = 4 if heads % 4 == 0 else 5
    Bn, U = heads // H, 2.0 ** -24
    r = torch.Generator(device="cuda").manual_seed(heads + dk + dv)
    rnd = lambda *s: torch.randn(s, generator=r, device="cuda")
    unit = lambda *s: torch.nn.functional.normalize(rnd(*s), dim=-1)
    dt = torch.float32 if io == "f32" else torch.bfloat16
    per = 2 if H == 4 else 1
    q, k, v = unit(Bn, H // per, dk).to(dt), unit(Bn, H // per, dk).to(dt), rnd(Bn, H, dv).to(dt)
    g, beta, S = -rnd(Bn, H).abs(), torch.sigmoid(2 * rnd(Bn, H)), rnd(Bn, H, dk, dv)
    g[0, 0] = -float("inf")
    print(f"[delta] step {io} {Bn} x {H} x {dk} x {dv}", flush=True)
    o1, S1 = B.deltarule_step(q, k, v, g, beta, S, scale=0.4, inplace=False)
    S2 = S.clone()
    o2, _ = B.deltarule_step(q, k, v, g, beta, S2, scale=0.4)
    o0, S0 = B.deltarule_step(q, k, v, g, beta, scale=0.4)
    torch.cuda.synchronize()
    half = 1.01 * 2.0 ** -8 if io == "bf16" else 2.0 ** -24
    for b in range(0, Bn, 64):
        n = slice(b, b + 64)
        Q, K = (x[n].double().repeat_interleave(per, 1) for x in (q, k))
        V, be, gam = v[n].double(), beta[n].double()[..., None], torch.exp(g[n].double())[..., None, None]
        left = lambda a, M: (a[..., None, :] @ M)[..., 0, :]
        for o, Sx, start in ((o1, S1, S), (o2, S2, S), (o0, S0, torch.zeros_like(S[:1, :1]).expand_as(S))):
            Sg = gam * start[n].double()
            u = be * (V - left(K, Sg))
            A = be * (V.abs() + left(K.abs(), Sg.abs()))
            ref, tol = Sg + K[..., None] * u[..., None, :], 16 * U * Sg.abs() + (dk + 64) * U * K.abs()[..., None] * A[..., None, :]
            assert bool(((Sx[n].double() - ref).abs() <= tol + U * ref.abs()).all())
            ro = 0.4 * left(Q, ref)
            Ao = 0.4 * (left(Q.abs(), Sg.abs()) + (Q * K).abs().sum(-1, keepdim=True) * A)
            assert bool(((o[n].double() - ro).abs() <= half * ro.abs() + (2 * dk + 128) * U * Ao).all())
