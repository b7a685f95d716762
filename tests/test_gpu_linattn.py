"""GPU parity of linear attention (linattn_fwd, linattn_step, linattn_bwd)
against the float64 oracle.

Tolerances, element by element.  Let A be the same operator applied to the
magnitudes of all inputs (every product then adds up, none cancels), N the
number of terms of a sum.
 * float32: a sum of N terms in any order is off by at most N 2^-24 A, its
   products and decays by a few 2^-24 A each (a decay e^{gn} whose exponent
   still matters has |gn| < 32, so it is off by 32 * 2^-23 relative).
 * bfloat16 inputs are exact; the state's copy that meets q, or the scores that
   meet v, may be rounded to bfloat16 once, 2^-8 A, the other of the two to 16
   bits, 2^-16 A; the output is rounded once, 2^-8 |o|.  The states are float32:
   2^-16 A is left for decayed values in parts.
"""
import numpy as np
import pytest
import torch

from oracle import ops as O
from xlstm_mlstm_matrix_amd import binding as B

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def make(io, Bn, H, T, dk, dv, seed=0, state=True, decay=None):
    r = np.random.default_rng(1000 + seed)
    t = lambda *s, std=1.0: torch.from_numpy(r.normal(0, std, s).astype(np.float32))
    d = {"q": t(Bn, H, T, dk), "k": t(Bn, H, T, dk, std=dk ** -0.5), "v": t(Bn, H, T, dv), "do": t(Bn, H, T, dv)}
    d = {n: x.to(DT[io]) for n, x in d.items()}
    if decay is None:
        decay = [-(2.0 ** (-8.0 * (h + 1) / H)) for h in range(H)]
    d["g"] = torch.tensor(decay, dtype=torch.float32)
    d["S0"] = t(Bn, H, dk, dv, std=0.3) if state else None
    d["dS"] = t(Bn, H, dk, dv, std=0.3) if state else None
    return d


def cu(d):
    return {n: None if x is None else x.cuda() for n, x in d.items()}


def mag(d):
    return {n: None if x is None else (x if n == "g" else x.abs()) for n, x in d.items()}


def check(x, ref, A, io, N, what, state=False):
    """Element by element, and the root mean square (2^-8 for bf16 results)."""
    x = x.detach().double().cpu().numpy()
    assert x.shape == ref.shape and np.all(np.isfinite(x)), what
    u = 2.0 ** -24
    if io == "f32":
        tol = (N + 64) * u * A + 1e-30
    elif state:
        tol = (2.0 ** -16 + (N + 64) * u) * A + 1e-30
    else:
        tol = HALF[io] * np.abs(ref) + (HALF[io] * 1.01 + 2.0 ** -15 + (N + 64) * u) * A + 1e-30
    bad = np.abs(x - ref) / tol
    rms = np.sqrt(np.mean((x - ref) ** 2) / max(np.mean(ref ** 2), 1e-60)) if x.size else 0.0
    print(f"[linattn] {what}: {bad.max():.3f} of the bound, rms {rms:.2e}", flush=True)
    assert bad.max() <= 1.0, (what, float(bad.max()))
    if io == "bf16" and not state:
        assert rms <= 2.0 ** -8, (what, rms)


def run_fwd(d, io, lengths=None, scale=1.0, what="", **kw):
    g = cu(d)
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    print(f"[linattn] fwd {what}", flush=True)
    o, S = B.linattn_fwd(g["q"], g["k"], g["v"], g["g"], g["S0"], lengths=ln, scale=scale, **kw)
    torch.cuda.synchronize()
    m = mag(d)
    ro, rS = O.linattn_forward(d["q"], d["k"], d["v"], d["g"], d["S0"], lengths, scale)
    Ao, AS = O.linattn_forward(m["q"], m["k"], m["v"], m["g"], m["S0"], lengths, abs(scale))
    N = d["q"].shape[2] + 2 * d["q"].shape[3]
    check(o, ro, Ao, io, N, what + " o")
    check(S, rS, AS, io, N, what + " S", state=True)
    return o, S


def run_bwd(d, io, lengths=None, scale=1.0, what=""):
    g = cu(d)
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    print(f"[linattn] bwd {what}", flush=True)
    got = B.linattn_bwd(g["q"], g["k"], g["v"], g["g"], g["do"], g["S0"], g["dS"], lengths=ln, scale=scale,
                        state_grad=True)
    torch.cuda.synchronize()
    m = mag(d)
    ref = O.linattn_backward(d["q"], d["k"], d["v"], d["g"], d["do"], d["S0"], d["dS"], lengths, scale)
    A = O.linattn_backward(m["q"], m["k"], m["v"], m["g"], m["do"], m["S0"], m["dS"], lengths, abs(scale))
    N = d["q"].shape[2] + 2 * max(d["q"].shape[3], d["v"].shape[3])
    for n, x, r, a in zip(("dq", "dk", "dv", "dS0"), got, ref, A):
        check(x, r, a, io, N, f"{what} {n}", state=n == "dS0")
    return got


SHAPES = [  # B, H, T, dk, dv
    (1, 1, 1, 16, 16), (2, 3, 5, 16, 48), (1, 2, 16, 32, 32), (2, 1, 63, 64, 64), (1, 2, 64, 64, 64),
    (1, 3, 65, 80, 112), (2, 2, 128, 128, 128), (1, 2, 129, 48, 208), (1, 1, 191, 256, 512),
    (1, 2, 200, 240, 272), (1, 1, 333, 128, 16), (1, 2, 97, 16, 512), (2, 2, 31, 256, 16),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_forward(io, shape):
    run_fwd(make(io, *shape, seed=sum(shape)), io, scale=shape[3] ** -0.5, what=f"{io} {shape}")


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_backward(io, shape):
    run_bwd(make(io, *shape, seed=sum(shape)), io, scale=shape[3] ** -0.5, what=f"{io} {shape}")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_long_sequence_of_few_heads(io):
    """Few cells and many chunks: the sequence is split into segments."""
    d = make(io, 1, 2, 1500, 64, 64, decay=[-0.002, -0.3])
    run_fwd(d, io, scale=0.125, what=f"{io} long")
    run_bwd(d, io, scale=0.125, what=f"{io} long")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_no_state_and_extreme_decays(io):
    """Decays of 0 (g = -inf), of almost 0, of exactly 1 (g = 0)."""
    d = make(io, 1, 5, 150, 32, 64, state=False, decay=[-float("inf"), -200.0, -1e30, 0.0, -1e-4])
    run_fwd(d, io, what=f"{io} extreme decays")
    run_bwd(d, io, what=f"{io} extreme decays")
    d = make(io, 1, 3, 70, 32, 64, decay=[-float("inf"), -87.0, 0.0])
    run_fwd(d, io, what=f"{io} extreme decays, state")
    run_bwd(d, io, what=f"{io} extreme decays, state")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T,lengths", [(130, [130, 64, 1, 0, 65, 129]), (40, [-3, 99, 16, 0, 40, 17]),
                                       (900, [900, 0, 449, 64, 513, 1])])
def test_padded_batch(io, T, lengths):
    """Rows behind a length are NaN in every input: nothing of them may show."""
    d = make(io, 6, 2, T, 64, 80, seed=T)
    clean = {n: x.clone() for n, x in d.items()}
    for b, n in enumerate(lengths):
        for name in ("q", "k", "v", "do"):
            d[name][b, :, min(max(n, 0), T):] = float("nan")
            clean[name][b, :, min(max(n, 0), T):] = 0
    g = cu(d)
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    o, S = run_fwd(clean, io, lengths, 0.125, what=f"{io} padded {T}")
    o2, S2 = B.linattn_fwd(g["q"], g["k"], g["v"], g["g"], g["S0"], lengths=ln, scale=0.125)
    assert torch.equal(o, o2) and torch.equal(S, S2)
    got = run_bwd(clean, io, lengths, 0.125, what=f"{io} padded {T}")
    got2 = B.linattn_bwd(g["q"], g["k"], g["v"], g["g"], g["do"], g["S0"], g["dS"], lengths=ln, scale=0.125,
                         state_grad=True)
    for a, b in zip(got, got2):
        assert torch.equal(a, b)
    for b, n in enumerate(lengths):
        for x in (o2, *got2[:3]):
            assert torch.count_nonzero(x[b, :, min(max(n, 0), T):]) == 0
        if n <= 0:
            assert torch.equal(S2[b], g["S0"][b]) and torch.equal(got2[3][b], g["dS"][b])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_strided_views_equal_dense(io):
    """Slices of one fused projection, token-major outputs, shared key heads."""
    Bn, H, T, dk, dv = 2, 4, 150, 64, 96
    r = torch.Generator(device="cuda").manual_seed(5)
    fused = torch.randn((Bn, T, H, 2 * dk + dv), generator=r, device="cuda").to(DT[io])
    q, k, v = (x.permute(0, 2, 1, 3) for x in fused.split([dk, dk, dv], -1))
    g = torch.tensor([-0.5, -0.1, -0.01, -2.0], device="cuda")
    o_tm = torch.full((Bn, T, H, dv), float("nan"), device="cuda", dtype=DT[io])
    o, S = B.linattn_fwd(q, k, v, g, scale=0.1, o=o_tm.permute(0, 2, 1, 3))
    od, Sd = B.linattn_fwd(q.contiguous(), k.contiguous(), v.contiguous(), g, scale=0.1)
    assert o.data_ptr() == o_tm.data_ptr()
    assert torch.equal(o, od) and torch.equal(S, Sd)
    do = torch.randn((Bn, T, H, dv), generator=r, device="cuda").to(DT[io]).permute(0, 2, 1, 3)
    buf = [torch.full((Bn, T, H, d), float("nan"), device="cuda", dtype=DT[io]) for d in (dk, dk, dv)]
    gr = B.linattn_bwd(q, k, v, g, do, scale=0.1, **{n: x.permute(0, 2, 1, 3) for n, x in zip(("dq", "dk", "dv"), buf)})
    gd = B.linattn_bwd(*(x.contiguous() for x in (q, k, v)), g, do.contiguous(), scale=0.1)
    for a, b in zip(gr, gd):
        assert torch.equal(a, b)
    # keys and values shared by all heads (stride 0): a gradient for each head
    k1, v1 = k[:, :1].expand(-1, H, -1, -1), v[:, :1].expand(-1, H, -1, -1)
    a, _ = B.linattn_fwd(q, k1, v1, g)
    b, _ = B.linattn_fwd(q, k1.contiguous(), v1.contiguous(), g)
    assert torch.equal(a, b)
    a = B.linattn_bwd(q, k1, v1, g, do)
    b = B.linattn_bwd(q, k1.contiguous(), v1.contiguous(), g, do)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("T", [150, 700])
def test_in_place_state_and_workspace(T):
    d = cu(make("bf16", 1, 2, T, 64, 64))
    o, S = B.linattn_fwd(d["q"], d["k"], d["v"], d["g"], d["S0"])
    S0 = d["S0"].clone()
    n = B.linattn_workspace_size(1, 2, T, 64, 64, B.BF16)
    ws = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN patterns
    o2, S2 = B.linattn_fwd(d["q"], d["k"], d["v"], d["g"], S0, S_T=S0, workspace=ws)
    assert S2 is S0 and torch.equal(o, o2) and torch.equal(S, S2)
    assert bool((ws[n:] == 0xFF).all())
    n = B.linattn_workspace_size(1, 2, T, 64, 64, B.BF16, True)
    ws = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    a = B.linattn_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], d["S0"], d["dS"], state_grad=True, workspace=ws)
    b = B.linattn_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], d["S0"], d["dS"], state_grad=True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert bool((ws[n:] == 0xFF).all())


def test_two_pieces_equal_one():
    """The state handed from one call to the next continues the sequence."""
    d = make("f32", 2, 2, 210, 64, 64)
    g = cu(d)
    o, S = run_fwd(d, "f32", what="whole")
    o1, S1 = B.linattn_fwd(g["q"][:, :, :77], g["k"][:, :, :77], g["v"][:, :, :77], g["g"], g["S0"])
    o2, S2 = B.linattn_fwd(g["q"][:, :, 77:], g["k"][:, :, 77:], g["v"][:, :, 77:], g["g"], S1)
    torch.testing.assert_close(torch.cat([o1, o2], 2), o, rtol=0, atol=2e-4)
    torch.testing.assert_close(S2, S, rtol=0, atol=2e-5)


STEPS = [(1, 1, 16, 16), (3, 5, 64, 64), (2, 3, 80, 112), (7, 2, 256, 512), (1, 3, 48, 208), (4, 2, 128, 128),
         (2, 1, 16, 512), (2, 2, 256, 16), (33, 8, 64, 64)]


@pytest.mark.parametrize("shape", STEPS, ids=str)
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("state", [True, False])
def test_step(io, shape, state):
    Bn, H, dk, dv = shape
    d = make(io, Bn, H, 1, dk, dv, seed=sum(shape), state=state)
    g, m = cu(d), mag(d)
    print(f"[linattn] step {io} {shape}", flush=True)
    o, S = B.linattn_step(g["q"][:, :, 0], g["k"][:, :, 0], g["v"][:, :, 0], g["g"], g["S0"], scale=0.3, inplace=False)
    torch.cuda.synchronize()
    ro, rS = O.linattn_forward(d["q"], d["k"], d["v"], d["g"], d["S0"], scale=0.3)
    Ao, AS = O.linattn_forward(m["q"], m["k"], m["v"], m["g"], m["S0"], scale=0.3)
    # float32 throughout, rounded once at the end
    x, u = o.double().cpu().numpy(), 2.0 ** -24
    assert np.all(np.abs(x - ro[:, :, 0]) <= HALF[io] * 1.01 * np.abs(ro[:, :, 0]) + (dk + 64) * u * Ao[:, :, 0])
    assert np.all(np.abs(S.double().cpu().numpy() - rS) <= 16 * u * AS)
    if state:   # in place, from strided rows
        fused = torch.cat([g["q"], g["k"], g["v"]], -1)[:, :, 0]
        q, k, v = fused.split([dk, dk, dv], -1)
        S1 = g["S0"].clone()
        o1, S2 = B.linattn_step(q, k, v, g["g"], S1, scale=0.3)
        assert S2 is S1 and torch.equal(S1, S) and torch.equal(o1, o)


def test_steps_continue_a_prefill():
    d = make("f32", 2, 3, 80, 64, 96)
    g = cu(d)
    o, S = run_fwd(d, "f32", what="steps")
    _, St = B.linattn_fwd(*(g[n][:, :, :70] for n in "qkv"), g["g"], g["S0"])
    for t in range(70, 80):
        ot, _ = B.linattn_step(*(g[n][:, :, t] for n in "qkv"), g["g"], St)
        torch.testing.assert_close(ot, o[:, :, t], rtol=0, atol=2e-4)
    torch.testing.assert_close(St, S, rtol=0, atol=2e-5)


def test_gradient_against_differences():
    """float32 call, directional differences taken with the float64 oracle."""
    d = make("f32", 1, 2, 90, 32, 32)
    g = cu(d)
    got = B.linattn_bwd(g["q"], g["k"], g["v"], g["g"], g["do"], g["S0"], g["dS"], state_grad=True)
    r = np.random.default_rng(3)
    x = {n: d[n].double().numpy() for n in ("q", "k", "v", "S0")}
    loss = lambda y: sum((a * d[n].double().numpy()).sum() for a, n in zip(
        O.linattn_forward(y["q"], y["k"], y["v"], d["g"], y["S0"]), ("do", "dS")))
    for n, gr in zip(("q", "k", "v", "S0"), got):
        e = r.normal(size=x[n].shape)
        h = 1e-4   # the loss is quadratic at most in one input: the difference is exact up to rounding
        num = (loss({**x, n: x[n] + h * e}) - loss({**x, n: x[n] - h * e})) / (2 * h)
        gn = gr.double().cpu().numpy()
        ana = (gn * e).sum()
        assert abs(num - ana) <= 1e-4 * np.sqrt((gn ** 2).sum() * (e ** 2).sum() / e.size) * np.sqrt(e.size), n


def test_other_stream_and_graph():
    """On a side stream, then captured once and replayed on changed inputs."""
    d = cu(make("bf16", 2, 2, 700, 64, 64))
    ref = B.linattn_fwd(d["q"], d["k"], d["v"], d["g"], d["S0"], scale=0.1)
    refb = B.linattn_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], d["S0"], d["dS"], scale=0.1, state_grad=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = B.linattn_fwd(d["q"], d["k"], d["v"], d["g"], d["S0"], scale=0.1)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = B.linattn_fwd(d["q"], d["k"], d["v"], d["g"], d["S0"], scale=0.1)
        gotb = B.linattn_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], d["S0"], d["dS"], scale=0.1, state_grad=True)
    for i in range(3):
        d["v"].mul_(-0.5)
        graph.replay()
        ref = B.linattn_fwd(d["q"], d["k"], d["v"], d["g"], d["S0"], scale=0.1)
        refb = B.linattn_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], d["S0"], d["dS"], scale=0.1, state_grad=True)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref + refb, got + gotb)), i


def test_refusals_of_the_binding():
    d = cu(make("bf16", 1, 2, 20, 32, 32))
    q, k, v, g = d["q"], d["k"], d["v"], d["g"]
    with pytest.raises(ValueError):
        B.linattn_fwd(q, k[:, :, :10], v, g)
    with pytest.raises(TypeError):
        B.linattn_fwd(q, k.float(), v, g)
    with pytest.raises(TypeError):
        B.linattn_fwd(q.half(), k.half(), v.half(), g)
    with pytest.raises(TypeError):
        B.linattn_fwd(q, k, v, g.double())
    with pytest.raises(ValueError):
        B.linattn_fwd(q, k, v.transpose(2, 3).contiguous().transpose(2, 3), g)
    with pytest.raises(TypeError):
        B.linattn_fwd(q, k, v, g, lengths=torch.tensor([3], device="cuda"))
    with pytest.raises(B.MlstmError):
        B.linattn_fwd(q, k, v, g, o=v)
    with pytest.raises(ValueError):
        B.linattn_bwd(q, k, v, g, d["do"], d["S0"][:, :1])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_step_of_states_larger_than_the_cache(io):
    """More than 256 MB of states take the streaming kernel; float64 on the device."""
    Bn, H, dk, dv = 37, 8, 256, 512
    r = torch.Generator(device="cuda").manual_seed(2)
    q, k = (torch.randn((Bn, H, dk), generator=r, device="cuda").to(DT[io]) for _ in range(2))
    v = torch.randn((Bn, H, dv), generator=r, device="cuda").to(DT[io])
    S = torch.randn((Bn, H, dk, dv), generator=r, device="cuda")
    g = torch.linspace(-2.0, 0.0, H, device="cuda")
    S64 = torch.exp(g.double())[:, None, None] * S.double() + k.double()[..., None] * v.double()[..., None, :]
    A = torch.exp(g.double())[:, None, None] * S.double().abs() + k.double().abs()[..., None] * v.double().abs()[..., None, :]
    ref = (q.double()[..., None] * S64).sum(-2) * 0.1
    oA = (q.double().abs()[..., None] * A).sum(-2) * 0.1
    o, S1 = B.linattn_step(q, k, v, g, S, scale=0.1)
    assert S1 is S
    u = 2.0 ** -24
    assert bool(((S1.double() - S64).abs() <= 16 * u * A).all())
    assert bool(((o.double() - ref).abs() <= HALF[io] * 1.01 * ref.abs() + (dk + 64) * u * oA).all())


@pytest.mark.parametrize("shape", [(1, 1, 1, 16, 16), (2, 2, 65, 64, 64), (1, 2, 700, 128, 128), (1, 1, 191, 256, 512),
                                   (2, 3, 130, 80, 112)], ids=str)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_outputs_without_state(io, shape):
    """Calls that hand out no state (their kernels carry it less finely)."""
    d = make(io, *shape, seed=7)
    g, m = cu(d), mag(d)
    s = shape[3] ** -0.5
    N = shape[2] + 2 * max(shape[3], shape[4])
    o = B.linattn_fwd(g["q"], g["k"], g["v"], g["g"], g["S0"], scale=s, return_state=False)
    assert torch.is_tensor(o)
    ro, _ = O.linattn_forward(d["q"], d["k"], d["v"], d["g"], d["S0"], scale=s)
    Ao, _ = O.linattn_forward(m["q"], m["k"], m["v"], m["g"], m["S0"], scale=s)
    check(o, ro, Ao, io, N, f"{io} {shape} o, no state")
    got = B.linattn_bwd(g["q"], g["k"], g["v"], g["g"], g["do"], g["S0"], g["dS"], scale=s)
    assert len(got) == 3
    ref = O.linattn_backward(d["q"], d["k"], d["v"], d["g"], d["do"], d["S0"], d["dS"], scale=s)
    A = O.linattn_backward(m["q"], m["k"], m["v"], m["g"], m["do"], m["S0"], m["dS"], scale=s)
    for n, x, r, a in zip(("dq", "dk", "dv"), got, ref, A):
        check(x, r, a, io, N, f"{io} {shape} {n}, no state")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_largest_token_stride(io):
    """Rows of 16 columns at the largest token stride, NaN between them: columns
    past the tensor's count as zeros, whatever a row's offset adds up to."""
    T, d = 40, 16
    ld = (1 << 22) - (4 if io == "f32" else 8)
    r = torch.Generator(device="cuda").manual_seed(9)
    buf = torch.full((T * ld,), float("nan"), device="cuda", dtype=DT[io])
    view = [torch.as_strided(buf, (1, 1, T, d), (0, 0, ld, 1), 64 * i) for i in range(4)]
    for x in view:
        x.copy_(torch.randn((1, 1, T, d), generator=r, device="cuda"))
    flat = [x.contiguous() for x in view]
    g = torch.tensor([-0.1], device="cuda")
    for a, b in zip(B.linattn_fwd(*view[:3], g), B.linattn_fwd(*flat[:3], g)):
        assert bool(torch.isfinite(b).all()) and torch.equal(a, b)
    for a, b in zip(B.linattn_bwd(*view[:3], g, view[3], state_grad=True),
                    B.linattn_bwd(*flat[:3], g, flat[3], state_grad=True)):
        assert bool(torch.isfinite(b).all()) and torch.equal(a, b)


@pytest.mark.parametrize("dv", [128, 208])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_step_of_many_narrow_states(io, dv):
    """More than 256 MB of states of 128 to 255 columns, a block that ends inside
    one among them; float64 on the device."""
    Bn, H, dk = 161, 16, 112
    r = torch.Generator(device="cuda").manual_seed(3)
    q, k = (torch.randn((Bn, H, dk), generator=r, device="cuda").to(DT[io]) for _ in range(2))
    v = torch.randn((Bn, H, dv), generator=r, device="cuda").to(DT[io])
    S = torch.randn((Bn, H, dk, dv), generator=r, device="cuda")
    assert S.numel() * 8 > 256 << 20
    g = torch.linspace(-2.0, 0.0, H, device="cuda")
    G = torch.exp(g.double())[:, None, None]
    kv = k.double()[..., None] * v.double()[..., None, :]
    S64, A = G * S.double() + kv, G * S.double().abs() + kv.abs()
    ref, oA = ((x[..., None] * y).sum(-2) for x, y in ((q.double(), S64), (q.double().abs(), A)))
    o, S1 = B.linattn_step(q, k, v, g, S)
    assert S1 is S
    u = 2.0 ** -24
    assert bool(((S1.double() - S64).abs() <= 16 * u * A).all())
    assert bool(((o.double() - ref).abs() <= HALF[io] * 1.01 * ref.abs() + (dk + 64) * u * oA).all())
