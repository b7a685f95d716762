"""Calls of the gated delta rule and of the norm and rotation at the ends of what their
header allows: the most heads, offsets past 2^32, calls in flight on two streams, replays of
captured calls, guard regions around every result.  References in float64 on the
device, or the same call on a part of the data."""
import pytest
import torch

from tests import deltarule_bounds as D
from tests.test_gpu_deltarule import DT, GRADS, cu, ints, make
from xlstm_mlstm_matrix_amd import binding as B

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def rnd(seed, shape, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def unit(seed, shape, dtype=torch.float32):
    x = rnd(seed, shape)
    return (x / x.norm(dim=-1, keepdim=True)).to(dtype)


def test_most_heads():
    """2^19 - 1 heads of one token: o = s beta (q.k) v and its gradients, float32."""
    n, d, s = (1 << 19) - 1, 16, 0.25
    q, k = unit(0, (1, n, 1, d)), unit(1, (1, n, 1, d))
    v, do = rnd(2, (1, n, 1, d)), rnd(3, (1, n, 1, d))
    g, beta = -rnd(4, (1, n, 1)).abs(), torch.sigmoid(rnd(5, (1, n, 1)))
    o = B.deltarule_fwd(q, k, v, g, beta, scale=s, return_state=False)
    dq, dk, dv, dg, db = B.deltarule_bwd(q, k, v, g, beta, do, scale=s)
    torch.cuda.synchronize()
    Q, K, V, DO, be = (x.double() for x in (q, k, v, do, beta[..., None]))
    qk, vd = (Q * K).sum(-1, keepdim=True), (V * DO).sum(-1, keepdim=True)
    aqk, avd = (Q * K).abs().sum(-1, keepdim=True), (V * DO).abs().sum(-1, keepdim=True)
    # sums of d products, products of two such sums, a few single roundings
    for x, ref, A in ((o, s * be * qk * V, aqk * V.abs()), (dq, s * be * vd * K, avd * K.abs()),
                      (dk, s * be * vd * Q, avd * Q.abs()), (dv, s * be * qk * DO, aqk * DO.abs()),
                      (db[..., None], s * qk * vd, aqk * avd)):
        assert bool(((x.double() - ref).abs() <= (2 * d + 64) * U * s * A).all())
    assert float(dg.abs().max()) <= (2 * d + 64) * U * float((aqk * avd).max())  # no state: exactly zero but for roundings


def test_long_sequence_past_32_bit_offsets():
    """2^22 + 5 tokens of 512 value columns: 4.3 GB of v, o and their gradients, in segments.
    With decays of e^-2 a token, the last tokens know only the 60 before them."""
    T, dk, dv, m = (1 << 22) + 5, 16, 512, 128
    q, k = unit(0, (1, 1, T, dk), torch.bfloat16), unit(1, (1, 1, T, dk), torch.bfloat16)
    v = torch.empty((1, 1, T, dv), dtype=torch.bfloat16, device="cuda")
    for t in range(0, T, 1 << 20):
        n = min(T - t, 1 << 20)
        v[0, 0, t:t + n] = rnd(100 + (t >> 20), (n, dv), torch.bfloat16)
    g = torch.full((1, 1, 1), -2.0, device="cuda").expand(1, 1, T)
    beta = torch.full((1, 1, 1), 0.5, device="cuda").expand(1, 1, T)
    cut = lambda x, a, b: x[:, :, a:b].contiguous()
    a = (q, k, v, g, beta)
    o, S = B.deltarule_fwd(*a, scale=0.25)
    close = lambda x, y, size: bool(((x.double() - y.double()).abs() <= 2.0 ** -7 * y.double().abs() + 2.0 ** -14 * size).all())
    for at in (T, T // 2 + 31, (1 << 21) + 50):     # ends of the data, and around 2^32 bytes of v
        ro, rS = B.deltarule_fwd(*(cut(x, at - m, at) for x in a), scale=0.25)
        assert close(o[:, :, at - 40:at], ro[:, :, -40:], 8), at
        if at == T:
            # sums of another split: float32, memory of a few tokens
            assert bool(((S - rS).abs() <= 512 * U * (1 + rS.abs())).all())
    del o
    got = B.deltarule_bwd(*a, v, scale=0.25)
    for lo, hi, take in ((0, m, slice(0, 40)), (T - m, T, slice(-40, None))):
        ref = B.deltarule_bwd(*(cut(x, lo, hi) for x in a), cut(v, lo, hi), scale=0.25)
        for x, y, size in zip(got, ref, (512, 512, 8, 512, 512)):
            x = x[:, :, lo:hi][:, :, take]
            assert close(x, y[:, :, take], size)


def test_two_streams_at_once():
    """Calls in flight on two streams, each with its own workspace, give what they give alone."""
    def inputs(seed):
        k = unit(seed, (1, 2, 3000, 64), torch.bfloat16)
        v, x = rnd(seed + 1, (1, 2, 3000, 64), torch.bfloat16), rnd(seed + 2, (1, 3000, 4, 64), torch.bfloat16)
        return k, v, -0.1 * rnd(seed + 3, (1, 2, 3000)).abs(), torch.sigmoid(rnd(seed + 4, (1, 2, 3000))), x

    def calls(k, v, g, beta, x):
        q, y = B.qknorm_fwd(x[:, :, :2].transpose(1, 2), x[:, :, 2:].transpose(1, 2), norm="l2")
        o, S = B.deltarule_fwd(q, k, v, g, beta, scale=0.2)
        back = B.deltarule_bwd(q, k, v, g, beta, o, dS_T=S, scale=0.2, state_grad=True)
        return (o, S, y) + back + B.qknorm_bwd(x[:, :, :2].transpose(1, 2), x[:, :, 2:].transpose(1, 2), back[0], back[1],
                                               norm="l2")

    x = [inputs(0), inputs(50)]
    ref = [calls(*a) for a in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for a, s in zip(x, streams):
            with torch.cuda.stream(s):
                got.append([calls(*a) for _ in range(3)])
        torch.cuda.synchronize()
        for runs, b in zip(got, ref):
            assert all(torch.equal(p, q) for r in runs for p, q in zip(r, b))


def test_replays_of_captured_calls():
    """A decode step with its norm and rotation, in place, and a whole training pass (forward and
    gradients in segments): every replay gives what the eager call gives."""
    x, v = rnd(0, (3, 1, 6, 64), torch.bfloat16), rnd(1, (3, 4, 96), torch.bfloat16)
    g, beta, S = -rnd(2, (3, 4)).abs(), torch.sigmoid(rnd(3, (3, 4))), rnd(4, (3, 4, 64, 96))
    f, pos = B.rope_frequencies(16, device="cuda")[0], torch.tensor([[5], [70], [100000]], dtype=torch.int32, device="cuda")
    eager = S.clone()

    def step(state):
        q, k = B.qknorm_fwd(x[:, :, :4].transpose(1, 2), x[:, :, 4:].transpose(1, 2), norm="l2", inv_freq=f, positions=pos)
        return B.deltarule_step(q[:, :2, 0], k[:, :, 0], v, g, beta, state, scale=0.3)[0]

    k2, v2 = unit(5, (1, 1, 700, 32), torch.bfloat16), rnd(6, (1, 1, 700, 32), torch.bfloat16)
    g2, b2 = -0.05 * rnd(7, (1, 1, 700)).abs(), torch.sigmoid(rnd(8, (1, 1, 700)))

    def train():
        o, ST = B.deltarule_fwd(k2, k2, v2, g2, b2)
        return (o, ST) + B.deltarule_bwd(k2, k2, v2, g2, b2, o)

    step(S.clone())
    train()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(S)
        out = train()
    for i in range(4):
        x.mul_(-0.75)
        v2.add_(0.25)
        pos.add_(1)
        graph.replay()
        ry, rout = step(eager), train()
        torch.cuda.synchronize()
        assert torch.equal(y, ry) and torch.equal(S, eager), i
        assert all(torch.equal(a, b) for a, b in zip(out, rout)), i


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 1, 2, 45, 48, 80), (1, 2, 2, 130, 64, 16), (1, 1, 1, 400, 16, 32)], ids=str)
def test_nothing_is_written_around_the_results(io, shape):
    """Every result inside a larger buffer of a fixed pattern, the workspace too."""
    Bn, Hk, H, T, dk, dv = shape
    d = make(io, *shape, seed=3)
    g = cu(d)
    lengths = ints([T] + [T // 3] * (Bn - 1))
    n, m = 4096, -12345.0
    store = []

    def guarded(size, dtype):
        numel = 1
        for s in size:
            numel *= s
        buf = torch.full((numel + 2 * n,), m, dtype=dtype, device="cuda")
        store.append((buf, numel))
        return buf[n:n + numel].view(size)

    a = [g[x] for x in ("q", "k", "v", "g", "beta")]
    dt = DT[io]
    plain = B.deltarule_fwd(*a, g["S0"], lengths=lengths, scale=0.3)
    back = B.deltarule_bwd(*a, g["do"], g["S0"], g["dS"], lengths=lengths, scale=0.3)
    need = [B.deltarule_workspace_size(Bn, Hk, H, T, dk, dv, int(io == "bf16"), b) for b in (False, True)]
    ws = [guarded((x // 4,), torch.float32) for x in need]
    o, S = B.deltarule_fwd(*a, g["S0"], lengths=lengths, scale=0.3, o=guarded((Bn, H, T, dv), dt),
                           S_T=guarded((Bn, H, dk, dv), torch.float32), workspace=ws[0])
    got = B.deltarule_bwd(*a, g["do"], g["S0"], g["dS"], lengths=lengths, scale=0.3, dq=guarded((Bn, Hk, T, dk), dt),
                          dk=guarded((Bn, Hk, T, dk), dt), dv=guarded((Bn, H, T, dv), dt),
                          dlog_decay=guarded((Bn, H, T), torch.float32), dbeta=guarded((Bn, H, T), torch.float32),
                          workspace=ws[1])
    torch.cuda.synchronize()
    for buf, numel in store:
        assert bool((buf[:n] == buf[0]).all()) and bool((buf[n + numel:] == buf[0]).all()) and float(buf[0]) == \
            float(torch.tensor(m, dtype=buf.dtype))
    for x, y in zip((o, S) + got, plain + back):
        assert torch.equal(x, y)


def draw(r):
    import numpy as np
    log = lambda lo, hi: int(round(np.exp(r.uniform(np.log(lo), np.log(hi + 0.49)))))
    Bn, Hk, per = log(1, 4), log(1, 5), int(r.choice([1, 1, 2, 3]))
    dk, dv = 16 * log(1, 16), 16 * log(1, 32)
    T = log(1, max(1, min(600, int(2.5e7 / (Bn * Hk * per * dk * dv) + 40))))
    return Bn, Hk, Hk * per, T, dk, dv


@pytest.mark.parametrize("seed", range(36))
def test_sweep(seed):
    """Head sizes, shared heads, tokens, lengths, decays, states, types drawn together."""
    import numpy as np
    from tests.test_gpu_deltarule import check
    r = np.random.default_rng(8700 + seed)
    io = ("f32", "bf16")[int(r.integers(2))]
    shape = draw(r)
    T = shape[3]
    lengths = [int(x) for x in r.integers(-1, T + 3, shape[0])] if r.random() < 0.5 else None
    d = make(io, *shape, seed=seed, state=bool(r.integers(2)), decay=float(2.0 ** -r.uniform(-2, 8)),
             alike=float(r.choice([0.0, 0.3, 1.0])))
    check(d, io, lengths, scale=shape[4] ** -0.5, what=f"{io} {shape} lengths {lengths} state {d['S0'] is not None}")


@pytest.mark.parametrize("seed", range(20))
def test_qknorm_sweep(seed):
    import numpy as np
    from tests.test_gpu_qknorm import run
    r = np.random.default_rng(8900 + seed)
    log = lambda lo, hi: int(round(np.exp(r.uniform(np.log(lo), np.log(hi + 0.49)))))
    d = int(r.choice([log(1, 512), 8 * log(1, 64)]))
    n = int(r.integers(0, d // 2 + 1))
    norm = ("rms", "l2", "none")[int(r.integers(3))]
    run(("f32", "bf16")[int(r.integers(2))], (log(1, 5), log(1, 60), log(1, 12), log(1, 12), d), n, norm,
        ("half", "pairs")[int(r.integers(2))], far=int(r.choice([0, 5000])), amp=float(r.choice([1.0, 1.2])), seed=seed,
        weight=bool(r.integers(2)), fused=bool(r.integers(2)))


def test_qknorm_past_32_bit_offsets():
    """2^20 + 3 tokens of 17 heads of 256 channels: 4.6e9 values, 9.1 GB."""
    T, H, d = (1 << 20) + 3, 17, 256
    x = torch.empty((1, T, H, d), dtype=torch.bfloat16, device="cuda")
    for t in range(0, T, 1 << 18):
        n = min(T - t, 1 << 18)
        x[0, t:t + n] = rnd(t >> 18, (n, H, d), torch.bfloat16)
    q, k = x[:, :, :16].transpose(1, 2), x[:, :, 16:].transpose(1, 2)
    f = B.rope_frequencies(64, device="cuda")[0]
    yq, yk = B.qknorm_fwd(q, k, norm="rms", inv_freq=f, layout="pairs")
    for t in (0, T // 2, T - 64):
        pos = torch.arange(t, t + 64, dtype=torch.int32, device="cuda")[None]
        one = B.qknorm_fwd(q[:, :, t:t + 64], k[:, :, t:t + 64], norm="rms", inv_freq=f, layout="pairs", positions=pos)
        assert torch.equal(yq[:, :, t:t + 64], one[0]) and torch.equal(yk[:, :, t:t + 64], one[1])
    dq, dk, _, dw = B.qknorm_bwd(q, k, yq, yk, norm="rms", inv_freq=f, layout="pairs", dq=yq, dk=yk)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(dw).all()) and bool((dk[0, 0, -64:].float().abs().amax(1) >= 0).all())
    assert bool(torch.isfinite(dq[0, :, -64:]).all())


def test_qknorm_most_rows():
    """2^31 - 1 rows, in place: two lanes a row are 2^32 threads, more than a launch takes."""
    T, d = (1 << 31) - 1, 9
    x = torch.full((1, 1, T, d), 2.0, dtype=torch.bfloat16, device="cuda")
    assert B.qknorm_fwd(x, norm="rms", yq=x) is x
    torch.cuda.synchronize()
    flat = x.view(-1)
    for i in range(0, flat.numel(), 1 << 32):
        assert bool((flat[i:i + (1 << 32)] == 1.0).all()), i
