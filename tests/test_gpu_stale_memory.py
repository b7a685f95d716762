"""No call's results depend on what earlier ones left behind: every operator after NaN in all of the
compute units' shared memory and in the memory that its workspaces and results are cut from,
against the same call after zeros, bit for bit.

Heads that fill no tile leave columns and rows of one unwritten; what is computed of those has
to reach no result, neither by a store nor as a factor of zero."""
import functools

import pytest
import torch

from xlstm_mlstm_matrix_amd import binding as B, inputs as I

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@functools.lru_cache(maxsize=None)
def filler(value):
    q = torch.full((1, 128, 128, 256), value, device="cuda")
    v = torch.full((1, 128, 128, 512), value, device="cuda")
    g = torch.full((1, 128, 128), value, device="cuda")
    return q, v, g


def leave(value):
    """``value`` (or what NaN makes of it) in the shared memory of every compute unit, and in free device
    memory, small blocks and large ones.  Float32 heads of 256 x 512: the forward has more workgroups of 157
    KB than there are units but zeros its first half at the end; the last kernel of the backward
    fills 118 KB from the start, also with more workgroups than units."""
    q, v, g = filler(value)
    B.deltarule_fwd(q, q, v, g, g)
    B.deltarule_bwd(q, q, v, g, g, v)
    torch.cuda.synchronize()
    blocks = [torch.full((n,), value, device="cuda") for n in [64 << 20] + [1 << 16] * 64 + [1 << 8] * 256]
    torch.cuda.synchronize()
    del blocks


def flat(out):
    if out is None:
        return []
    if isinstance(out, torch.Tensor):
        return [out]
    return [x for o in out for x in flat(o)]


def check(call, what):
    print(f"[stale] {what}", flush=True)
    results = []
    for value in (0.0, float("nan"), float("nan")):
        leave(value)
        out = flat(call())
        torch.cuda.synchronize()
        results.append([x.clone() for x in out])
    for i, xs in enumerate(zip(*results)):
        assert bool(torch.isfinite(xs[0]).all()), (what, i)
        for x in xs[1:]:
            assert torch.equal(x, xs[0]), (what, i, int((x != xs[0]).sum()))


def rnd(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s, dt="f32", std=1.0: (torch.randn(s, generator=g, device="cuda") * std).to(DT[dt])


DIMS = [(16, 16), (48, 80), (64, 64), (80, 48), (112, 144), (128, 128), (240, 400), (256, 512), (16, 512), (176, 208)]


@pytest.mark.parametrize("dk,dv", DIMS, ids=str)
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("state", [False, True])
def test_cell(io, dk, dv, state):
    r = rnd(dk + dv)
    Bn, H, T = 2, 24, 75
    q, k = (r(Bn, H, T, dk, dt=io, std=dk ** -0.5) for _ in range(2))
    v, o, dh = (r(Bn, H, T, dv, dt=io) for _ in range(3))
    i, f = r(Bn, H, T), -r(Bn, H, T).abs()
    st = (r(Bn, H, dk, dv), r(Bn, H, dk), r(Bn, H)) if state else (None, None, None)
    for chunk in (32, 64):
        check(lambda: B.fwd_chunkwise(q, k, v, i, f, o, *st, chunk=chunk), f"{io} {dk} x {dv} forward {chunk} state {state}")
    check(lambda: B.bwd_chunkwise(q, k, v, i, f, o, dh, *st, state_grad=True), f"{io} {dk} x {dv} backward state {state}")
    first = [x[:, :, 0].contiguous() for x in (q, k, v, i, f, o)]
    check(lambda: B.step(*first, *st, inplace=False), f"{io} {dk} x {dv} step state {state}")


@pytest.mark.parametrize("dk,dv", [(16, 48), (64, 64), (80, 112), (128, 128), (240, 400), (256, 512)], ids=str)
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("variant", ["fused", "segscan"])
def test_cell_schedules(io, dk, dv, variant):
    """Both schedules of the forward, every chunk length that a size takes."""
    r = rnd(dk + dv + 1)
    H, T = 3, 600
    q, k = (r(1, H, T, dk, dt=io, std=dk ** -0.5) for _ in range(2))
    v, o = (r(1, H, T, dv, dt=io) for _ in range(2))
    i, f = r(1, H, T), -r(1, H, T).abs()
    st, ran = (r(1, H, dk, dv), r(1, H, dk), r(1, H)), 0
    for chunk in (16, 32, 64, 128, 256):
        try:
            B.workspace_size(1, H, T, dk, dv, chunk, int(io == "bf16"), variant)
        except B.MlstmError:
            continue
        check(lambda: B.fwd_chunkwise(q, k, v, i, f, o, *st, chunk=chunk, variant=variant),
              f"{io} {dk} x {dv} {variant} {chunk}")
        ran += 1
    assert ran


@pytest.mark.parametrize("pairs", [1, 2, 7])
@pytest.mark.parametrize("dk,dv", [(16, 16), (16, 80), (64, 48), (48, 144), (256, 208)], ids=str)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gradients_of_few_pairs(io, dk, dv, pairs):
    """Few workgroups: each pass may meet a compute unit that none of those before it has used."""
    r = rnd(dk + dv + pairs)
    for T in (1, 20, 64, 200):
        q, k = (r(1, pairs, T, dk, dt=io, std=dk ** -0.5) for _ in range(2))
        v, o, dh = (r(1, pairs, T, dv, dt=io) for _ in range(3))
        i, f = r(1, pairs, T), -r(1, pairs, T).abs()
        for st in ((None, None, None), (r(1, pairs, dk, dv), r(1, pairs, dk), r(1, pairs))):
            check(lambda: B.bwd_chunkwise(q, k, v, i, f, o, dh, *st, state_grad=True),
                  f"{io} {dk} x {dv} backward of {pairs} x {T}, state {st[0] is not None}")


@pytest.mark.parametrize("dk,dv", DIMS, ids=str)
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 75, 600])
def test_operators(io, dk, dv, T):
    r = rnd(dk + dv + T)
    for H in (3, 40) if T < 600 else (2,):
        q, k = (torch.nn.functional.normalize(r(2, H, T, dk), dim=-1).to(DT[io]) for _ in range(2))
        v, do = (r(2, H, T, dv, dt=io) for _ in range(2))
        g, beta, decay = -0.1 * r(2, H, T).abs(), torch.sigmoid(r(2, H, T)), -0.1 * r(H).abs()
        S, D = r(2, H, dk, dv), r(2, H, dk, dv)
        n = torch.tensor([T, T // 3], dtype=torch.int32, device="cuda")
        what = f"{io} {dk} x {dv}, {H} heads of {T}"
        for s, d, ln in ((S, D, n), (None, None, None)):
            check(lambda: B.linattn_fwd(q, k, v, decay, s, lengths=ln), what + " linattn")
            check(lambda: B.linattn_bwd(q, k, v, decay, do, s, d, lengths=ln, state_grad=s is not None), what + " linattn_bwd")
            check(lambda: B.deltarule_fwd(q, k, v, g, beta, s, lengths=ln), what + " deltarule")
            check(lambda: B.deltarule_bwd(q, k, v, g, beta, do, s, d, lengths=ln, state_grad=s is not None),
                  what + " deltarule_bwd")
        check(lambda: B.deltarule_bwd(q[:, :1], k[:, :1], v, g, beta, do, S, D, lengths=n), what + " deltarule_bwd, shared")
        check(lambda: B.deltarule_fwd(q, k, v, g, beta, return_state=False), what + " deltarule, no state")
        a = [x[:, :, 0] for x in (q, k, v)]
        check(lambda: B.linattn_step(*a, decay, S, inplace=False), what + " linattn_step")
        check(lambda: B.deltarule_step(*a, g[:, :, 0], beta[:, :, 0], S, inplace=False), what + " deltarule_step")


@pytest.mark.parametrize("d,n", [(1, 0), (33, 8), (64, 32), (96, 36), (128, 64), (257, 100), (512, 256)])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_norms(io, d, n):
    r = rnd(d)
    f = B.rope_frequencies(n, device="cuda")[0] if n else None
    w, b = 1 + 0.1 * r(d), 0.1 * r(4, d)
    for T in (1, 333):
        q, k, dq, dk = (r(2, h, T, d, dt=io) for h in (4, 2, 4, 2))
        check(lambda: B.qknorm_fwd(q, k, w, w, inv_freq=f), f"{io} {d} qknorm of {T}")
        check(lambda: B.qknorm_bwd(q, k, dq, dk, w, w, inv_freq=f), f"{io} {d} qknorm_bwd of {T}")
        x, dy = r(2, T, 4, d, dt=io), r(2, T, 4, d, dt=io)
        wt = 1 + 0.1 * r(4, d)
        for over in ("token", "sequence"):
            if over == "token" and d == 1:
                continue
            y, mean, rstd = B.groupnorm_fwd(x, wt, b, act="silu", over=over)
            check(lambda: B.groupnorm_fwd(x, wt, b, act="silu", over=over), f"{io} {d} groupnorm of {T} {over}")
            check(lambda: B.groupnorm_bwd(x, dy, mean, rstd, wt, b, act="silu", over=over),
                  f"{io} {d} groupnorm_bwd of {T} {over}")


@pytest.mark.parametrize("override", [dict(name="layer_small"), dict(name="layer_small", d_qk=48, d_v=80, d_model=96),
                                      dict(name="layer_7b_bf16", B=1, T=150, d_model=512, H=2),
                                      dict(name="layer_7b_bf16", B=2, T=70, d_model=192, H=3, d_qk=48, d_v=112)], ids=str)
def test_layer(override):
    d = {k: v.cuda() if v is not None else None for k, v in I.gen_layer(I.layer_workload(**override)).items()}
    names = ("x", "W_q", "W_k", "W_v", "W_o", "W_i", "W_f", "b_q", "b_k", "b_v", "b_o", "b_i", "b_f", "C0", "n0", "m0")
    for chunk in (32, 64):
        check(lambda: B.layer_fwd(*(d[n] for n in names), chunk=chunk), f"{override} {chunk}")


@pytest.mark.parametrize("override", [dict(name="slstm_small", T=40), dict(name="slstm_bf16", T=40, B=3, H=2),
                                      dict(name="slstm_bf16", T=9, B=1, H=1, d=48)], ids=str)
def test_slstm(override):
    d = {k: v.cuda() if v is not None else None for k, v in I.gen_slstm(I.slstm_workload(**override)).items()}
    check(lambda: B.slstm_fwd(d["gx"], d["R"], d["c0"], d["n0"], d["m0"], d["h0"]), str(override))
