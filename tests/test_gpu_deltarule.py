"""GPU parity of the gated delta rule (deltarule_fwd, deltarule_step, deltarule_bwd)
with the recurrence in float64; tolerances are derived in deltarule_bounds.py."""
import numpy as np
import pytest
import torch

from oracle import ops as O
from tests import deltarule_bounds as D
from xlstm_mlstm_matrix_amd import binding as B

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
INF = float("inf")
GRADS = ("dq", "dk", "dv", "dg", "dbeta", "dS0")


def make(io, Bn, Hk, H, T, dk, dv, seed=0, state=True, decay=0.2, alike=0.3):
    """Unit queries and keys with a common part (``alike``), strengths in (0, 1)."""
    r = np.random.default_rng(2000 + seed)
    t = lambda *s, std=1.0: torch.from_numpy(r.normal(0, std, s).astype(np.float32))

    def unit(*s):
        x = t(*s) + alike * 3.0 * t(*s[:2], 1, s[3])
        return x / x.norm(dim=-1, keepdim=True)

    d = {"q": unit(Bn, Hk, T, dk), "k": unit(Bn, Hk, T, dk), "v": t(Bn, H, T, dv), "do": t(Bn, H, T, dv)}
    d = {n: x.to(DT[io]) for n, x in d.items()}
    d["g"] = -decay * torch.nn.functional.softplus(t(Bn, H, T))
    d["beta"] = torch.sigmoid(2.0 * t(Bn, H, T))
    d["S0"] = t(Bn, H, dk, dv, std=0.3) if state else None
    d["dS"] = t(Bn, H, dk, dv, std=0.3) if state else None
    return d


def cu(d):
    return {n: None if x is None else x.cuda() for n, x in d.items()}


def ints(lengths):
    return None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")


def check(d, io, lengths=None, scale=1.0, what="", backward=True, g=None, clean=None):
    """Forward and gradients of the inputs d (g: the device copies, clean: what the
    reference sees)."""
    g = cu(d) if g is None else g
    clean = d if clean is None else clean
    print(f"[delta] {what}", flush=True)
    args = [g[n] for n in ("q", "k", "v", "g", "beta")]
    o, S = B.deltarule_fwd(*args, g["S0"], lengths=ints(lengths), scale=scale)
    torch.cuda.synchronize()
    w = D.sweep(clean if backward else {**clean, "do": None}, lengths, scale)
    D.check(w, {"o": o, "S": S}, io, what)
    if not backward:
        return o, S
    got = B.deltarule_bwd(*args, g["do"], g["S0"], g["dS"], lengths=ints(lengths), scale=scale, state_grad=True)
    torch.cuda.synchronize()
    D.check(w, dict(zip(GRADS, got)), io, what)
    return (o, S) + got


SHAPES = [  # B, Hk, H, T, dk, dv
    (1, 1, 1, 1, 16, 16), (2, 3, 3, 5, 16, 48), (1, 2, 2, 16, 32, 32), (2, 1, 1, 31, 64, 64), (1, 2, 4, 32, 64, 64),
    (1, 3, 3, 33, 80, 112), (2, 1, 2, 64, 128, 128), (1, 2, 2, 65, 48, 208), (1, 1, 1, 97, 256, 512),
    (1, 1, 3, 100, 240, 272), (1, 1, 1, 161, 128, 16), (1, 2, 2, 97, 16, 512), (2, 2, 2, 17, 256, 16),
    (1, 1, 2, 129, 64, 128), (1, 1, 1, 200, 96, 144),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_shapes(io, shape):
    check(make(io, *shape, seed=sum(shape)), io, scale=shape[4] ** -0.5, what=f"{io} {shape}")


def test_the_reference_is_the_oracle():
    """The bounds' own sweep against the oracle, with shared heads and lengths."""
    d = make("f32", 2, 2, 4, 9, 16, 16)
    n = [9, 4]
    w = D.sweep(d, n, 0.5)
    a = [d[x] for x in ("q", "k", "v", "g", "beta")]
    o, S = O.deltarule_forward(*a, d["S0"], n, 0.5)
    back = O.deltarule_backward(*a, d["do"], d["S0"], d["dS"], n, 0.5)
    for x, y in zip([w[n] for n in ("o", "S") + GRADS], (o, S) + back):
        assert np.allclose(x.numpy(), y, rtol=1e-10, atol=1e-11)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_no_state(io):
    d = make(io, 2, 2, 2, 70, 32, 64, state=False)
    what = f"{io} no state"
    got = check(d, io, scale=0.2, what=what)
    g = cu(d)
    a = [g[x] for x in ("q", "k", "v", "g", "beta")]
    one = B.deltarule_fwd(*a, scale=0.2, return_state=False)
    less = B.deltarule_bwd(*a, g["do"], scale=0.2)
    torch.cuda.synchronize()
    D.check(D.sweep(d, None, 0.2), {"o": one, **dict(zip(GRADS, less))}, io, what + " returned")
    assert len(less) == 5 and len(got) == 8


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_extreme_gates(io):
    """Decays of 0 (-inf) and of 1 (0), far below float32's range, strengths of 0, 1 and 2."""
    d = make(io, 1, 6, 6, 150, 32, 64, seed=5, decay=0.05)
    r = np.random.default_rng(6)
    d["g"][0, 0] = 0.0
    d["g"][0, 1, ::7] = -INF
    d["g"][0, 2, ::5] = -1e30
    d["g"][0, 3] = torch.from_numpy(r.choice([-200.0, -1e4, -0.01], 150).astype(np.float32))
    d["g"][0, 4, 40] = -INF
    d["beta"][0, 0] = torch.from_numpy(r.choice([0.0, 1.0, 2.0], 150).astype(np.float32))
    d["beta"][0, 5] = 0.0
    got = check(d, io, scale=0.3, what=f"{io} extreme gates")
    zero = (d["g"] == -INF).cuda()
    assert bool((got[5][zero] == 0).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_same_key_again_and_again(io):
    """All keys of a head alike, strength 1: the inverse's entries come from sums
    of large terms if it is not solved row by row."""
    d = make(io, 1, 2, 2, 96, 64, 64, seed=7, decay=0.0)
    d["k"][0, 0] = d["k"][0, 0, :1]
    d["beta"][0, 0] = 1.0
    d["k"][0, 1, 1::2] = -d["k"][0, 1, :1]
    d["k"][0, 1, ::2] = d["k"][0, 1, :1]
    d["beta"][0, 1] = 1.9
    check(d, io, scale=0.125, what=f"{io} one key")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T,lengths", [(130, [130, 64, 1, 0, 65, 129]), (40, [-3, 99, 16, 0, 40, 17]),
                                       (300, [300, 0, 149, 32, 97, 1])])
def test_padded_batch(io, T, lengths):
    """Rows behind a length are NaN in every input: nothing of them may show."""
    d = make(io, 6, 1, 2, T, 64, 80, seed=T)
    clean = {n: x.clone() for n, x in d.items()}
    for b, n in enumerate(lengths):
        for name in ("q", "k", "v", "do", "g", "beta"):
            d[name][b, :, min(max(n, 0), T):] = float("nan")
            clean[name][b, :, min(max(n, 0), T):] = 0
    o, S, dq, dk, dv, dg, db, dS0 = check(d, io, lengths, 0.125, f"{io} padded {T}", clean=clean)
    for b, n in enumerate(lengths):
        n = min(max(n, 0), T)
        for x in (o, dq, dk, dv, dg, db):
            assert bool((x[b, :, n:] == 0).all())
        if n == 0:
            assert torch.equal(S[b].cpu(), d["S0"][b]) and torch.equal(dS0[b].cpu(), d["dS"][b])


def rows(t, pad=16):
    """The same [B, H, T, d] values as a view of wider token-major rows, NaN around them."""
    Bn, H, T, d = t.shape
    x = torch.full((Bn, T, H, d + pad), float("nan"), dtype=t.dtype, device="cuda")
    v = x[..., pad:].permute(0, 2, 1, 3)
    v.copy_(t)
    return v


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_strided_views(io):
    """Token-major rows, gates of a [B, T, 2 H + 1] projection, results into views."""
    d = make(io, 2, 2, 4, 75, 64, 96, seed=8)
    g = cu(d)
    dense = check(d, io, scale=0.2, what=f"{io} dense")
    s = {n: rows(g[n]) if n in ("q", "k", "v", "do") else g[n] for n in g}
    gates = torch.full((2, 75, 9), float("nan"), device="cuda")
    s["g"], s["beta"] = gates[..., 1:5].transpose(1, 2), gates[..., 5:].transpose(1, 2)
    s["g"].copy_(g["g"])
    s["beta"].copy_(g["beta"])
    a = [s[n] for n in ("q", "k", "v", "g", "beta")]
    o = rows(torch.zeros_like(g["v"]))
    S = g["S0"].clone()
    B.deltarule_fwd(*a, S, scale=0.2, o=o, S_T=S)
    out = [rows(torch.zeros_like(g[n])) for n in ("q", "k", "v")]
    dg, db = (torch.zeros((2, 75, 5), device="cuda")[..., 1:].transpose(1, 2) for _ in range(2))
    got = B.deltarule_bwd(*a, s["do"], g["S0"], g["dS"], scale=0.2, state_grad=True, dq=out[0], dk=out[1],
                          dv=out[2], dlog_decay=dg, dbeta=db)
    torch.cuda.synchronize()
    assert got[3] is dg and got[4] is db
    for x, y in zip((o, S) + got, dense):
        assert torch.equal(x, y)


def test_repeated_inputs():
    """Rows repeated over the batch and gates over time (stride 0)."""
    d = make("bf16", 1, 2, 2, 50, 32, 32, seed=9)
    g = cu(d)
    wide = {n: x.expand(3, *x.shape[1:]) if x is not None else None for n, x in g.items()}
    wide["g"] = torch.full((1, 2, 1), -0.1, device="cuda").expand(3, 2, 50)
    full = {n: x.contiguous() if x is not None else None for n, x in wide.items()}
    call = lambda w: B.deltarule_bwd(*(w[n] for n in ("q", "k", "v", "g", "beta", "do")), full["S0"], full["dS"]) \
        + B.deltarule_fwd(*(w[n] for n in ("q", "k", "v", "g", "beta")), full["S0"])
    for x, y in zip(call(wide), call(full)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_continued_from_a_state(io):
    """Two calls in a row against one, and the step against both."""
    d = make(io, 2, 2, 4, 83, 64, 96, seed=10)
    g = cu(d)
    names = ("q", "k", "v", "g", "beta")
    check(d, io, scale=0.3, what=f"{io} whole", backward=False)
    cut = lambda a, b: [g[n][:, :, a:b] for n in names]
    S = g["S0"].clone()
    o1, S = B.deltarule_fwd(*[x.contiguous() for x in cut(0, 45)], S, scale=0.3, S_T=S)
    o2, S = B.deltarule_fwd(*cut(45, 82), S, scale=0.3)
    o3, S = B.deltarule_step(*[x[:, :, 0] for x in cut(82, 83)], S, scale=0.3)
    torch.cuda.synchronize()
    w = D.sweep({**d, "do": None}, None, 0.3)
    D.check(w, {"o": torch.cat([o1, o2, o3[:, :, None]], 2), "S": S}, io, f"{io} in parts")


STEPS = [(1, 1, 1, 16, 16), (3, 8, 8, 64, 64), (2, 2, 6, 80, 48), (5, 1, 2, 128, 128), (2, 3, 3, 256, 512),
         (1, 2, 2, 240, 272), (2, 1, 1, 16, 512), (1, 1, 4, 256, 16), (7, 4, 4, 112, 208)]


@pytest.mark.parametrize("shape", STEPS, ids=str)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_step(io, shape):
    Bn, Hk, H, dk, dv = shape
    for state in (True, False):
        d = make(io, Bn, Hk, H, 1, dk, dv, seed=sum(shape), state=state)
        if Bn > 1:
            d["g"][1] = -INF
            d["beta"][0] = 0.0
        g = cu(d)
        a = [g[n][:, :, 0] for n in ("q", "k", "v", "g", "beta")]
        print(f"[delta] {io} step {shape} state {state}", flush=True)
        o, S = B.deltarule_step(*a, g["S0"], scale=0.4, inplace=False)
        torch.cuda.synchronize()
        D.check(D.sweep({**d, "do": None}, None, 0.4), {"o": o[:, :, None], "S": S}, io, f"{io} step {shape}")
        if state:
            o2, S2 = B.deltarule_step(*a, g["S0"], scale=0.4)
            assert S2 is g["S0"] and torch.equal(S2, S) and torch.equal(o2, o)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_long_sequence_of_few_heads(io):
    check(make(io, 1, 1, 2, 1500, 64, 64, seed=11, decay=0.02), io, scale=0.125, what=f"{io} long")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 700, 240, 32), (1, 1, 3, 600, 96, 176), (2, 1, 2, 530, 16, 64)], ids=str)
def test_segments(io, shape):
    """Few heads and many chunks in segments: sizes that fill no tile, lengths that end in
    every segment, strong and weak decays."""
    d = make(io, *shape, seed=13, decay=0.01)
    d["g"][:, -1] *= 30.0
    T = shape[3]
    lengths = None if shape[0] == 1 else [T, 97]
    if lengths is not None:
        for n in ("q", "k", "v", "do", "g", "beta"):
            d[n][1, :, 97:] = 0
    check(d, io, lengths, scale=0.2, what=f"{io} segments {shape}")
    if shape[0] == 1:
        check({**d, "S0": None, "dS": None}, io, [T - 290], scale=0.2, what=f"{io} segments {shape} short", backward=False)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_state_in_place_over_segments(io):
    """S_T over S0 where the sequence runs in segments, against separate tensors; an empty
    sequence among them keeps its state."""
    d = make(io, 3, 1, 1, 900, 64, 128, seed=14, decay=0.01)
    g = cu(d)
    a = [g[n] for n in ("q", "k", "v", "g", "beta")]
    n = ints([900, 0, 333])
    o, S = B.deltarule_fwd(*a, g["S0"], lengths=n, scale=0.2)
    for _ in range(5):
        state = g["S0"].clone()
        o2, S2 = B.deltarule_fwd(*a, state, lengths=n, scale=0.2, S_T=state)
        torch.cuda.synchronize()
        assert S2 is state and torch.equal(o, o2) and torch.equal(S, S2)
    assert torch.equal(S[1], g["S0"][1])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gradients_over_segments_of_a_padded_batch(io):
    """Sequences that end in the last segment, the first, a middle one and before any
    token, of heads that share queries and keys."""
    lengths = [700, 20, 333, 0]
    d = make(io, 4, 1, 2, 700, 48, 32, seed=15, decay=0.01)
    for i, n in enumerate(lengths):
        for name in ("q", "k", "v", "do", "g", "beta"):
            d[name][i, :, n:] = 0
    check(d, io, lengths, scale=0.2, what=f"{io} padded segments")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_segments_without_a_state(io):
    """Segments where no state is given or asked for: fewer parts of the states between
    them in bfloat16."""
    d = make(io, 1, 1, 2, 640, 64, 96, seed=16, state=False, decay=0.01)
    g = cu(d)
    a = [g[x] for x in ("q", "k", "v", "g", "beta")]
    o = B.deltarule_fwd(*a, scale=0.2, return_state=False)
    got = B.deltarule_bwd(*a, g["do"], scale=0.2)
    torch.cuda.synchronize()
    D.check(D.sweep(d, None, 0.2), {"o": o, **dict(zip(GRADS, got))}, io, f"{io} segments, no state")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_extreme_gates_over_segments(io):
    """Decays of 0 and 1 and reflections (strength 2 and a unit key) in sequences of segments,
    one that forgets everything in each segment and one that forgets nothing."""
    d = make(io, 1, 4, 4, 600, 32, 64, seed=17, decay=0.02)
    d["g"][0, 0] = 0.0
    d["beta"][0, 0] = 2.0
    d["g"][0, 1, ::60] = -INF
    d["g"][0, 2, 300:] = -1e30
    d["beta"][0, 3] = 0.0
    got = check(d, io, scale=0.3, what=f"{io} extreme gates, segments")
    assert bool((got[5][(d["g"] == -INF).cuda()] == 0).all())


def test_gradients_are_the_differences():
    """float32 gradients against differences of the forward's own results: a change of
    2^-7 in a random direction, twice, leaves third-order terms, 2^-14 of the loss's
    curvature in that direction."""
    d = make("f32", 1, 1, 2, 40, 16, 16, seed=12)
    g = cu(d)
    names = ("q", "k", "v", "g", "beta")
    gen = torch.Generator(device="cuda").manual_seed(1)
    grads = B.deltarule_bwd(*(g[n] for n in names), g["do"], g["S0"], g["dS"], scale=0.3, state_grad=True)

    def loss(x):
        o, S = B.deltarule_fwd(*(x[n] for n in names), x["S0"], scale=0.3)
        return float((o.double() * g["do"].double()).sum() + (S.double() * g["dS"].double()).sum())

    for n, gr in zip(names + ("S0",), grads):
        v = torch.randn(g[n].shape, generator=gen, device="cuda") * 0.1
        h = 2.0 ** -7
        num = (loss({**g, n: g[n] + h * v}) - loss({**g, n: g[n] - h * v})) / (2 * h)
        far = (loss({**g, n: g[n] + 2 * h * v}) - loss({**g, n: g[n] - 2 * h * v})) / (4 * h)
        want = float((gr.double() * v.double()).sum())
        # Richardson: |far - num| is 3 times num's own third-order error; sums of 640 terms of order 1
        # in float32, over 2 h
        tol = 1.1 * abs(far - num) / 3 + 640 * 2.0 ** -24 * 4 / (2 * h) * float((g["do"].abs()).mean())
        assert abs(num - want) <= tol, (n, num, want, tol)
