"""Calls of the operators at the ends of what their header allows: the most heads,
offsets past 2^32 elements or bytes, calls in flight on two streams, steps replayed
from a graph.  References in float64 on the device, or the same call on a part of
the data."""
import pytest
import torch

from xlstm_mlstm_matrix_amd import binding as B

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def rnd(seed, shape, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def test_most_heads():
    """2^19 - 1 heads of one token: o = s (q.k) v and its gradients, float32."""
    n, d, s = (1 << 19) - 1, 256, 0.25
    q, k, v, do = (rnd(i, (1, n, 1, d)) for i in range(4))
    g = torch.full((n,), -0.1, device="cuda")
    o = B.linattn_fwd(q, k, v, g, scale=s, return_state=False)
    dq, dk, dv = B.linattn_bwd(q, k, v, g, do, scale=s)
    torch.cuda.synchronize()
    for i in range(0, n, 1 << 16):
        Q, K, V, DO = (x[0, i:i + (1 << 16), 0].double() for x in (q, k, v, do))
        dot = lambda a, b: ((a * b).sum(-1, keepdim=True) * s, (a * b).abs().sum(-1, keepdim=True) * s)
        (qk, aqk), (dv_, adv) = dot(Q, K), dot(DO, V)
        for x, ref, A in ((o, qk * V, aqk * V.abs()), (dq, dv_ * K, adv * K.abs()), (dk, dv_ * Q, adv * Q.abs()),
                          (dv, qk * DO, aqk * DO.abs())):
            # a sum of d products in any order, a few roundings more
            assert bool(((x[0, i:i + (1 << 16), 0].double() - ref).abs() <= (d + 64) * U * A).all())


def test_most_heads_step():
    n, d = (1 << 19) - 1, 32
    q, k, v = (rnd(i, (n, 1, d)) for i in range(3))
    S = rnd(4, (n, 1, d, d))
    g = torch.tensor([-0.5], device="cuda")
    o, S1 = B.linattn_step(q, k, v, g, S, inplace=False)
    torch.cuda.synchronize()
    for i in range(0, n, 1 << 16):
        p = slice(i, i + (1 << 16))
        kv, G = k[p].double()[..., None] * v[p].double()[..., None, :], torch.exp(g.double())
        ref, A = G * S[p].double() + kv, G * S[p].double().abs() + kv.abs()
        assert bool(((S1[p].double() - ref).abs() <= 16 * U * A).all())
        ro, Ao = ((a.double()[..., None] * b).sum(-2) for a, b in ((q[p], ref), (q[p].abs(), A)))
        assert bool(((o[p].double() - ro).abs() <= (d + 64) * U * Ao).all())


def test_long_sequence_past_32_bit_offsets():
    """2^23 + 5 tokens of 512 value columns: 8.6 GB of v and of o.  With decays of e^-2
    a token, the last ones know only the 60 before them: they equal a short call's,
    up to what two sums in another order differ by."""
    T, dk, dv, m = (1 << 23) + 5, 16, 512, 100
    q, k = (rnd(i, (1, 1, T, dk), torch.bfloat16) for i in range(2))
    v = torch.empty((1, 1, T, dv), dtype=torch.bfloat16, device="cuda")
    for t in range(0, T, 1 << 20):
        n = min(T - t, 1 << 20)
        v[0, 0, t:t + n] = rnd(100 + (t >> 20), (n, dv), torch.bfloat16)
    g = torch.tensor([-2.0], device="cuda")
    tail = lambda x, at: x[:, :, at - m:at].contiguous()
    o, S = B.linattn_fwd(q, k, v, g, scale=0.25)
    for at in (T, T // 2, (1 << 22) + 50):     # ends of the data, and around 2^32 bytes of v
        ro, rS = B.linattn_fwd(tail(q, at), tail(k, at), tail(v, at), g, scale=0.25)
        a, b = o[0, 0, at - 40:at].double(), ro[0, 0, m - 40:].double()
        # one rounding apart, and 2^-14 of the sums' terms (|q| |k| |v| of 16 columns)
        assert bool(((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -14 * 64).all()), at
        if at == T:
            assert bool(((S - rS).abs() <= 64 * U * (1 + rS.abs()) * 16).all())
    del o
    # backward: from the last token back, so the first ones know only those behind them
    do, v0 = v, v[:, :, :m].contiguous()
    dq, dkk, dvv = B.linattn_bwd(q, k, v, g, do, scale=0.25)
    r = B.linattn_bwd(q[:, :, :m].contiguous(), k[:, :, :m].contiguous(), v0, g, v0, scale=0.25)
    e = B.linattn_bwd(tail(q, T), tail(k, T), tail(v, T), g, tail(v, T), scale=0.25)
    for x, a, b in zip((dq, dkk, dvv), r, e):
        for y, z in ((x[0, 0, :40], a[0, 0, :40]), (x[0, 0, -40:], b[0, 0, -40:])):
            # terms are sums of 512 products for dq and dk
            assert bool(((y.double() - z.double()).abs() <= 2.0 ** -7 * z.double().abs() + 2.0 ** -14 * 2048).all())


@pytest.mark.parametrize("over", ["token", "sequence"])
def test_norm_past_32_bit_offsets(over):
    """2^20 + 3 positions of 4112 channels: 4.3e9 values, 8.6 GB."""
    S, G, D = (1 << 20) + 3, 8, 514
    x = torch.empty((1, S, G, D), dtype=torch.bfloat16, device="cuda")
    for p in range(0, S, 1 << 17):
        n = min(S - p, 1 << 17)
        x[0, p:p + n] = rnd(p >> 17, (n, G, D), torch.bfloat16) + 0.5
    w, b = rnd(91, (G, D)), rnd(92, (G, D))
    y, m, r = B.groupnorm_fwd(x, w, b, act="silu", over=over)
    torch.cuda.synchronize()
    if over == "sequence":
        s1 = s2 = 0
        for p in range(0, S, 1 << 17):
            X = x[0, p:p + (1 << 17)].double()
            s1, s2 = s1 + X.sum((0, 2)), s2 + (X * X).sum((0, 2))
        mu = s1 / (S * D)
        rs = (s2 / (S * D) - mu * mu + 1e-5).rsqrt()
        # sums of blocks of positions: a few hundred roundings at most
        assert bool(((m[0].double() - mu).abs() <= 512 * U).all()) and bool(((r[0].double() / rs - 1).abs() <= 512 * U).all())
    for p in (0, S // 2, S - 64):
        X = x[0, p:p + 64].double()
        if over == "token":
            mu = X.mean(-1, keepdim=True)
            rs = (((X - mu) ** 2).mean(-1, keepdim=True) + 1e-5).rsqrt()
        else:
            mu, rs = mu.reshape(1, G, 1), rs.reshape(1, G, 1)
        z = (X - mu) * rs * w.double() + b.double()
        ref = z * torch.sigmoid(z)
        assert bool(((y[0, p:p + 64].double() - ref).abs() <= 2.0 ** -8 * 1.01 * ref.abs() + 2.0 ** -12).all()), p
    del y
    dx, dw, db = B.groupnorm_bwd(x, x, m, r, w, b, act="silu", over=over)
    torch.cuda.synchronize()
    if over == "token":
        for p in (0, S // 2, S - 64):
            one = B.groupnorm_bwd(x[:, p:p + 64].contiguous(), x[:, p:p + 64].contiguous(), m[:, p:p + 64].contiguous(),
                                  r[:, p:p + 64].contiguous(), w, b, act="silu")
            assert torch.equal(dx[:, p:p + 64], one[0]), p
    else:
        assert bool(torch.isfinite(dx[0, -64:]).all()) and bool((dx[0, -64:].float().abs().amax((1, 2)) > 0).all())
    assert bool(torch.isfinite(dw).all()) and bool(torch.isfinite(db).all())


def test_two_streams_at_once():
    """Calls in flight on two streams, each with its own workspace, give what they
    give alone."""
    def inputs(seed):
        q, k, v, do = (rnd(seed + i, (1, 2, 3000, 64), torch.bfloat16) for i in range(4))
        return q, k, v, torch.tensor([-0.05, -0.4], device="cuda"), do

    def calls(q, k, v, g, do):
        o, S = B.linattn_fwd(q, k, v, g, scale=0.1)
        y, m, r = B.groupnorm_fwd(o.transpose(1, 2), over="sequence", act="gelu")
        dx, _, _ = B.groupnorm_bwd(o.transpose(1, 2), do.transpose(1, 2), m, r, over="sequence", act="gelu")
        return (o, S, y, dx) + B.linattn_bwd(q, k, v, g, dx.transpose(1, 2), scale=0.1)

    x = [inputs(0), inputs(50)]
    ref = [calls(*a) for a in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for a, s in zip(x, streams):
            with torch.cuda.stream(s):
                got.append([calls(*a) for _ in range(4)])
        torch.cuda.synchronize()
        for runs, b in zip(got, ref):
            assert all(torch.equal(p, q) for r in runs for p, q in zip(r, b))


def test_steps_replayed_from_a_graph():
    """A captured step with its head norm, in place: each replay advances the state."""
    q, k = (rnd(i, (3, 4, 64), torch.bfloat16) for i in range(2))
    v, w = rnd(2, (3, 4, 96), torch.bfloat16), rnd(3, (4, 96))
    g = torch.tensor([-0.5, -0.1, -0.01, 0.0], device="cuda")
    S = rnd(4, (3, 4, 64, 96))
    eager = S.clone()
    step = lambda state: B.groupnorm_fwd(B.linattn_step(q, k, v, g, state, scale=0.1)[0][:, None], w, act="silu",
                                         return_stats=False)
    step(S.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(S)
    for i in range(4):
        q.mul_(-0.75)
        graph.replay()
        ref = step(eager)
        torch.cuda.synchronize()
        assert torch.equal(y, ref) and torch.equal(S, eager), i
