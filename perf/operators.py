"""Workloads of linear attention with a decay for each head and of group norm
with an activation: their inputs, their plain forms in elementary torch
operations, and the work that each cannot do without.

Linear attention (state S [d_qk, d_v] of each head, g its log decay):

    S_t = e^g S_{t-1} + k_t v_t^T,    o_t = scale * q_t^T S_t

as a whole sequence (``prefill``), a single token (``step``) and the gradients
of a sequence (``backward``).  Group norm of x [N, S, G, D]: each group is
normalised over its D channels at each position (``over="token"``, the norm of
a head) or over all S positions too (``over="sequence"``), scaled, shifted and
passed through an activation; forward (``norm``) and gradients
(``norm_grad``).
"""
import math

import torch

own = False   # True: the library's kernels; False: the plain forms below

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases

def _seq(name, op, B, H, T, dk, dv, io, ragged=False, token_major=False, state=False):
    c = {"op": op, "B": B, "H": H, "T": T, "dk": dk, "dv": dv, "io": io, "ragged": ragged,
         "token_major": token_major, "state": state}
    return {"name": name, **c} if name else c


def _step(name, B, H, dk, dv, io):
    c = {"op": "step", "B": B, "H": H, "dk": dk, "dv": dv, "io": io}
    return {"name": name, **c} if name else c


def _norm(name, op, N, S, G, D, io, act, over, head_major=False):
    c = {"op": op, "N": N, "S": S, "G": G, "D": D, "io": io, "act": act, "over": over,
         "head_major": head_major}
    return {"name": name, **c} if name else c


def listed():
    return [
        # a short prompt continued from a state, float32: latency counts
        _seq("prefill_short_f32", "prefill", 1, 4, 37, 64, 64, "f32", state=True),
        # a padded batch of prompts read straight out of a fused projection
        # (token-major rows), lengths from the full 2000 down to an empty one
        _seq("prefill_padded_bf16", "prefill", 6, 16, 2000, 128, 128, "bf16", ragged=True,
             token_major=True, state=True),
        # the sequence shape of the library's own 7B-layer prefill workload
        _seq("prefill_7b_bf16", "prefill", 8, 8, 4096, 256, 512, "bf16"),
        # one long document: few heads in flight, many chunks in a row
        _seq("prefill_long_bf16", "prefill", 1, 8, 32768, 128, 128, "bf16", state=True),
        # single tokens of a small and of the library's decode batch
        _step("step_small_bf16", 3, 8, 64, 64, "bf16"),
        _step("step_batch_bf16", 256, 8, 256, 512, "bf16"),
        # gradients at the library's float32 training shape, carried state included
        _seq("backward_small_f32", "backward", 4, 4, 1024, 64, 64, "f32", state=True),
        # a training step's gradients of one layer of 16 heads of 128
        _seq("backward_layer_bf16", "backward", 4, 16, 4096, 128, 128, "bf16", token_major=True),
        # the head norm behind the 7B-layer cell: head-major h to token-major rows
        _norm("norm_heads_bf16", "norm", 8, 4096, 8, 512, "bf16", "none", "token", head_major=True),
        # feature maps, channels last, 10 channels a group (not a vector's width)
        _norm("norm_map_f32", "norm", 8, 1024, 32, 10, "f32", "silu", "sequence"),
        # gradients of the head norm of a layer of 16 heads of 128
        _norm("norm_grad_heads_bf16", "norm_grad", 4, 4096, 16, 128, "bf16", "silu", "token"),
        # gradients over whole sequences
        _norm("norm_grad_map_bf16", "norm_grad", 6, 2500, 32, 40, "bf16", "gelu", "sequence"),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "step", "backward", "backward", "norm", "norm_grad"])
    io = rng.choice(["f32", "bf16", "bf16"])
    if op in ("prefill", "backward"):
        dk = 16 * _logint(rng, 1, 16)
        dv = 16 * _logint(rng, 1, 32)
        B, H = _logint(rng, 1, 16), _logint(rng, 1, 32)
        # tokens so that the case's products and rows stay below the largest listed ones'
        cap = min(2.5e10 / (dk * dv), 3e8 / (2 * dk + 2 * dv)) if op == "prefill" \
            else min(4e9 / (dk * dv), 1.8e8 / (4 * dk + 3 * dv))
        cap /= B * H * (8 if io == "f32" else 1)
        T = _logint(rng, 1, max(1, min(16384, int(cap))))
        return _seq(None, op, B, H, T, dk, dv, io, ragged=B > 1 and rng.random() < 0.5,
                    token_major=rng.random() < 0.5, state=rng.random() < 0.5)
    if op == "step":
        dk = 16 * _logint(rng, 1, 16)
        dv = 16 * _logint(rng, 1, 32)
        H = _logint(rng, 1, 32)
        B = _logint(rng, 1, max(1, min(512, int(2.6e8 / (H * dk * dv)))))
        return _step(None, B, H, dk, dv, io)
    over = rng.choice(["token", "sequence"])
    act = rng.choice(["none", "silu", "gelu"])
    G = _logint(rng, 1, 64)
    D = 16 * _logint(rng, 1, 32) if over == "token" else _logint(rng, 1, 256)
    N = _logint(rng, 1, 16)
    S = _logint(rng, 1, max(1, min(8192, int(2.5e7 / (N * G * D)))))
    return _norm(None, op, N, S, G, D, io, act, over, head_major=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs

def _lengths(case):
    """Tokens of each sequence of a padded batch: the first is full, the last empty."""
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return [T] * B
    return [T * (B - 1 - b) // (B - 1) for b in range(B)]


def _gen(seed, dev="cuda"):
    g = torch.Generator(device=dev)
    g.manual_seed(0x51A7 + 7919 * int(seed))
    return g


def _rand(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=g.device) * std).to(dtype)


def _heads(g, case, d, dtype, std=1.0):
    """A [B, H, T, d] tensor, dense or as a view of token-major [B, T, H, d] rows."""
    B, H, T = case["B"], case["H"], case["T"]
    if case["token_major"]:
        return _rand(g, (B, T, H, d), dtype, std).transpose(1, 2)
    return _rand(g, (B, H, T, d), dtype, std)


def _log_decay(H):
    """Geometric rates over the heads: from a memory of a few tokens to one of hundreds."""
    return torch.tensor([-(2.0 ** (-8.0 * (h + 1) / H)) for h in range(H)], dtype=torch.float32,
                        device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    dt = _DT[case["io"]]
    op = case["op"]
    st = {"case": case}
    if op in ("prefill", "backward"):
        B, H, dk, dv = (case[x] for x in ("B", "H", "dk", "dv"))
        st["q"] = _heads(g, case, dk, dt)
        st["k"] = _heads(g, case, dk, dt, dk ** -0.5)
        st["v"] = _heads(g, case, dv, dt)
        st["g"] = _log_decay(H)
        st["scale"] = dk ** -0.5
        st["S0"] = _rand(g, (B, H, dk, dv), torch.float32, 0.1) if case["state"] else None
        st["lengths"] = (torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
                         if case["ragged"] else None)
        if op == "backward":
            st["do"] = _heads(g, case, dv, dt)
            st["dS"] = _rand(g, (B, H, dk, dv), torch.float32, 0.1) if case["state"] else None
    elif op == "step":
        B, H, dk, dv = (case[x] for x in ("B", "H", "dk", "dv"))
        st["q"] = _rand(g, (B, H, dk), dt)
        st["k"] = _rand(g, (B, H, dk), dt, dk ** -0.5)
        st["v"] = _rand(g, (B, H, dv), dt)
        st["g"] = _log_decay(H)
        st["scale"] = dk ** -0.5
        st["S"] = _rand(g, (B, H, dk, dv), torch.float32, 0.1)
        st["S_out"] = torch.empty_like(st["S"])
    else:
        N, S, G, D = (case[x] for x in ("N", "S", "G", "D"))

        def rows(mean=0.0):
            if case["head_major"]:
                t = torch.randn((N, G, S, D), generator=g, device="cuda").transpose(1, 2)
            else:
                t = torch.randn((N, S, G, D), generator=g, device="cuda")
            return (t + mean).to(dt)

        st["x"] = rows(0.25)
        st["w"] = 1.0 + 0.2 * torch.randn((G, D), generator=g, device="cuda")
        st["b"] = 0.2 * torch.randn((G, D), generator=g, device="cuda")
        if op == "norm_grad":
            st["dy"] = rows()
            st["mean"], st["rstd"] = _moments(st["x"].float(), case["over"])
    return st


# ---------------------------------------------------------------- plain forms

_EPS = 1e-5
_CHUNK = 128


def _chunked(q, k, v, g, S, p_scale, in_scale, up_scale, shift):
    """Float32 chunked linear attention of dense [B, H, T, .] rows from the
    state S: scores scaled by p_scale, the carried state's read-out by
    in_scale, its update by up_scale; with shift = 1 the carried state has
    already decayed once (the reverse direction)."""
    B, H, T, dk = q.shape
    out = torch.empty((B, H, T, v.shape[-1]), dtype=torch.float32, device=q.device)
    for c in range(0, T, _CHUNK):
        qc, kc, vc = q[:, :, c:c + _CHUNK], k[:, :, c:c + _CHUNK], v[:, :, c:c + _CHUNK]
        n = qc.shape[2]
        t = torch.arange(n, device=q.device, dtype=torch.float32)
        dist = t[:, None] - t[None, :]
        dec = torch.exp(g[:, None, None] * dist.clamp(min=0.0)) * (dist >= 0)
        a = torch.matmul(qc, kc.transpose(-1, -2)) * dec * p_scale
        fade = torch.exp(g[:, None] * (t + 1.0 - shift))[:, :, None]
        out[:, :, c:c + n] = torch.matmul(a, vc) + torch.matmul(qc * fade, S) * in_scale
        keep = torch.exp(g[:, None] * (n - 1.0 + shift - t))[:, :, None]
        S = torch.exp(g * n)[:, None, None] * S + torch.matmul((kc * keep).transpose(-1, -2), vc) * up_scale
    return out, S


def _valid(st, T):
    """[B, 1, T, 1] mask of the tokens before each sequence's length (None: all)."""
    if st["lengths"] is None:
        return None
    return (torch.arange(T, device="cuda")[None, :] < st["lengths"][:, None])[:, None, :, None]


def _float_rows(st, *names):
    """Contiguous float32 copies, tokens behind a sequence's length zeroed."""
    T = st["q"].shape[2]
    m = _valid(st, T)
    out = []
    for n in names:
        x = st[n].float().contiguous()
        out.append(x if m is None else torch.where(m, x, torch.zeros((), device="cuda")))
    return out


def _state32(S, like, dk, dv):
    return S if S is not None else torch.zeros(like.shape[:2] + (dk, dv), device="cuda")


def _end_state(k, v, g, S, fade, keep, up_scale):
    """e^{g fade} S + up_scale * sum_t e^{g keep_t} k_t v_t^T; rows with keep < 0 do not count.
    fade [B], keep [B, T]."""
    w = torch.exp(g[None, :, None] * keep.clamp(min=0)[:, None, :]) * (keep >= 0)[:, None, :]
    out = torch.matmul((k * w[..., None]).transpose(-1, -2), v) * up_scale
    return out + torch.exp(g[None, :] * fade[:, None])[..., None, None] * S


def _plain_prefill(st):
    q, k, v = _float_rows(st, "q", "k", "v")
    S0 = _state32(st["S0"], q, k.shape[-1], v.shape[-1])
    L, s, g = st["lengths"], st["scale"], st["g"]
    o, S = _chunked(q, k, v, g, S0, s, s, 1.0, 0.0)
    if L is not None:   # the state after each sequence's own last token
        t = torch.arange(q.shape[2], device="cuda")[None, :]
        S = _end_state(k, v, g, S0, L, L[:, None] - 1 - t, 1.0)
    return o.to(st["q"].dtype), S


def _plain_step(st):
    S = torch.exp(st["g"])[None, :, None, None] * st["S"] \
        + st["k"].float()[..., None] * st["v"].float()[..., None, :]
    o = (st["q"].float()[..., None] * S).sum(-2) * st["scale"]
    return o.to(st["q"].dtype), S


def _plain_backward(st):
    q, k, v, do = _float_rows(st, "q", "k", "v", "do")
    dk, dv = q.shape[-1], v.shape[-1]
    g, s, L = st["g"], st["scale"], st["lengths"]
    S0 = _state32(st["S0"], q, dk, dv)
    dS = _state32(st["dS"], q, dk, dv)
    tr = lambda x: x.transpose(-1, -2).contiguous()
    # dq reads the forward's states
    dq, _ = _chunked(do, v, k, g, tr(S0), s, s, 1.0, 0.0)
    # dk, dv read the gradient of the state, carried from the last token back;
    # in a padded batch dS enters each sequence at its own last token
    carried = dS if L is None else torch.zeros_like(dS)
    rq, rk, rv, rdo = (x.flip(2) for x in (q, k, v, do))
    dvv, dS0 = _chunked(rk, rq, rdo, g, carried, s, 1.0, s, 1.0)
    dkk, _ = _chunked(rv, rdo, rq, g, tr(carried), s, 1.0, s, 1.0)
    dvv, dkk = dvv.flip(2), dkk.flip(2)
    if L is not None:
        t = torch.arange(q.shape[2], device="cuda")[None, :]
        fade = torch.exp(g[None, :, None] * (L[:, None] - 1 - t).clamp(min=0)[:, None, :])[..., None]
        dvv = dvv + torch.matmul(k * fade, dS)
        dkk = dkk + torch.matmul(v * fade, tr(dS))
        dS0 = _end_state(q, do, g, dS, L, torch.where(t < L[:, None], t + 1, -1), s)
    dt = st["q"].dtype
    out = (dq.to(dt), dkk.to(dt), dvv.to(dt))
    return out + (dS0,) if st["dS"] is not None else out


def _moments(x, over):
    """Mean and 1/sqrt(var + eps) over the channels, or channels and positions."""
    dims = (3,) if over == "token" else (1, 3)
    mu = x.mean(dims, keepdim=True)
    var = ((x - mu) ** 2).mean(dims, keepdim=True)
    r = torch.rsqrt(var + _EPS)
    if over == "token":
        return mu[..., 0].contiguous(), r[..., 0].contiguous()
    return mu[:, 0, :, 0].contiguous(), r[:, 0, :, 0].contiguous()


def _act(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return z


def _dact(z, act):
    if act == "silu":
        sg = 1.0 / (1.0 + torch.exp(-z))
        return sg * (1.0 + z * (1.0 - sg))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) \
            + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    return torch.ones_like(z)


def _spread(t, over):
    return t[..., None] if over == "token" else t[:, None, :, None]


def _plain_norm(st):
    c = st["case"]
    x = st["x"].float()
    mean, rstd = _moments(x, c["over"])
    z = (x - _spread(mean, c["over"])) * _spread(rstd, c["over"]) * st["w"] + st["b"]
    return _act(z, c["act"]).to(st["x"].dtype), mean, rstd


def _plain_norm_grad(st):
    c = st["case"]
    x, dy = st["x"].float(), st["dy"].float()
    r = _spread(st["rstd"], c["over"])
    xh = (x - _spread(st["mean"], c["over"])) * r
    dz = dy * _dact(xh * st["w"] + st["b"], c["act"])
    dims = (3,) if c["over"] == "token" else (1, 3)
    dxh = dz * st["w"]
    dx = r * (dxh - dxh.mean(dims, keepdim=True) - xh * (dxh * xh).mean(dims, keepdim=True))
    return dx.to(st["x"].dtype), (dz * xh).sum((0, 1)), dz.sum((0, 1))


_PLAIN = {"prefill": _plain_prefill, "step": _plain_step, "backward": _plain_backward,
          "norm": _plain_norm, "norm_grad": _plain_norm_grad}


# ---------------------------------------------------------------- one pass

def run(st):
    c = st["case"]
    op = c["op"]
    if not own:
        return _PLAIN[op](st)
    from xlstm_mlstm_matrix_amd import binding as B
    if op == "prefill":
        return B.linattn_fwd(st["q"], st["k"], st["v"], st["g"], st["S0"], lengths=st["lengths"],
                             scale=st["scale"])
    if op == "step":
        return B.linattn_step(st["q"], st["k"], st["v"], st["g"], st["S"], scale=st["scale"],
                              S_out=st["S_out"])
    if op == "backward":
        return B.linattn_bwd(st["q"], st["k"], st["v"], st["g"], st["do"], st["S0"], st["dS"],
                             lengths=st["lengths"], scale=st["scale"], state_grad=st["dS"] is not None)
    if op == "norm":
        return B.groupnorm_fwd(st["x"], st["w"], st["b"], eps=_EPS, act=c["act"], over=c["over"])
    return B.groupnorm_bwd(st["x"], st["dy"], st["mean"], st["rstd"], st["w"], st["b"], act=c["act"],
                           over=c["over"])


# ---------------------------------------------------------------- work

def work(case):
    """Each input read once, each output written once; multiply-adds of the recurrent form."""
    op = case["op"]
    e = 4 if case["io"] == "f32" else 2
    if op == "step":
        n, d = case["B"] * case["H"], case["dk"] * case["dv"]
        return {"bytes": n * (8 * d + e * (2 * case["dk"] + 2 * case["dv"])), "flops": n * 5 * d}
    if op in ("prefill", "backward"):
        H, dk, dv = case["H"], case["dk"], case["dv"]
        rows = sum(_lengths(case)) * H
        all_rows = case["B"] * case["T"] * H
        state = case["B"] * H * dk * dv * 4
        if op == "prefill":
            # q, k, v of the real tokens, o of all rows; the state in and out
            b = e * (rows * (2 * dk + dv) + all_rows * dv) + state * (2 if case["state"] else 1)
            return {"bytes": b, "flops": rows * 4 * dk * dv}
        b = e * (rows * (2 * dk + 2 * dv) + all_rows * (2 * dk + dv))
        return {"bytes": b + state * (3 if case["state"] else 0), "flops": rows * 10 * dk * dv}
    n = case["N"] * case["S"] * case["G"] * case["D"]
    groups = case["N"] * case["G"] * (case["S"] if case["over"] == "token" else 1)
    par = case["G"] * case["D"] * 8
    if op == "norm":
        return {"bytes": 2 * n * e + 8 * groups + par, "flops": 10 * n}
    return {"bytes": 3 * n * e + 8 * groups + 2 * par, "flops": 20 * n}


# ---------------------------------------------------------------- exact values

def exact(case, seed):
    """The recurrences token by token, and the norm from its definition, in float64."""
    op = case["op"]
    st = prepare(case, seed)
    if op == "step":
        g = st["g"].double()
        S = torch.exp(g).reshape(1, -1, 1, 1) * st["S"].double()
        S = S + st["k"].double().unsqueeze(-1) * st["v"].double().unsqueeze(-2)
        return (st["q"].double().unsqueeze(-2) @ S).squeeze(-2) * st["scale"], S
    if op in ("prefill", "backward"):
        return _exact_sequence(case, st)
    return _exact_norm(case, st)


def _exact_sequence(case, st):
    B, H, T, dk, dv = (case[x] for x in ("B", "H", "T", "dk", "dv"))
    # each token reads and writes the whole state, in float64
    if T * (1e-4 + B * H * dk * dv * 16 / 1.5e12) * (1 if case["op"] == "prefill" else 3) > 20.0:
        return None
    s = st["scale"]
    gam = torch.exp(st["g"].double()).reshape(1, H, 1, 1)
    L = _lengths(case)
    # sequences in order of their length, so those still running are the first ones
    order = sorted(range(B), key=lambda b: -L[b])
    perm = torch.tensor(order, device="cuda")
    live = [sum(1 for b in range(B) if L[b] > t) for t in range(T)]
    z = lambda d: torch.zeros((T, B, H, d), dtype=torch.float64, device="cuda")
    tok = lambda n: st[n].double()[perm].permute(2, 0, 1, 3).contiguous()       # [T, B, H, d]
    start = lambda n: (torch.zeros((B, H, dk, dv), dtype=torch.float64, device="cuda")
                       if st[n] is None else st[n].double()[perm])
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(B, device="cuda")
    back = lambda x: x.permute(1, 2, 0, 3)[inv]
    q, k, v = tok("q"), tok("k"), tok("v")
    S = start("S0")
    if case["op"] == "prefill":
        o = z(dv)
        for t in range(T):
            n = live[t]
            if n == 0:
                break
            Sn = S[:n]
            Sn.mul_(gam).addcmul_(k[t, :n, :, :, None], v[t, :n, :, None, :])
            o[t, :n] = (q[t, :n, :, None, :] @ Sn)[:, :, 0] * s
        return back(o), S[inv]
    do = tok("do")
    dq, dkk, dvv = z(dk), z(dk), z(dv)
    for t in range(T):
        n = live[t]
        if n == 0:
            break
        Sn = S[:n]
        Sn.mul_(gam).addcmul_(k[t, :n, :, :, None], v[t, :n, :, None, :])
        dq[t, :n] = (Sn @ do[t, :n, :, :, None])[..., 0] * s
    D = start("dS")
    for t in range(T - 1, -1, -1):
        n = live[t]
        if n == 0:
            continue
        Dn = D[:n]
        Dn.addcmul_(q[t, :n, :, :, None], do[t, :n, :, None, :], value=s)
        dkk[t, :n] = (Dn @ v[t, :n, :, :, None])[..., 0]
        dvv[t, :n] = (k[t, :n, :, None, :] @ Dn)[:, :, 0]
        Dn.mul_(gam)
    out = (back(dq), back(dkk), back(dvv))
    return out + (D[inv],) if st["dS"] is not None else out


def _exact_norm(case, st):
    N, S, G, D = (case[x] for x in ("N", "S", "G", "D"))
    # [groups, members]: one row for each set of values normalised together
    if case["over"] == "token":
        rows = lambda t: t.double().reshape(N * S * G, D)
        par = lambda p: p.double().expand(N, S, G, D).reshape(N * S * G, D)
        unrows = lambda t: t.reshape(N, S, G, D)
        stat = lambda t: t.reshape(N, S, G)
    else:
        rows = lambda t: t.double().permute(0, 2, 1, 3).reshape(N * G, S * D)
        par = lambda p: p.double().expand(N, S, G, D).permute(0, 2, 1, 3).reshape(N * G, S * D)
        unrows = lambda t: t.reshape(N, G, S, D).permute(0, 2, 1, 3)
        stat = lambda t: t.reshape(N, G)
    x, w, b = rows(st["x"]), par(st["w"]), par(st["b"])
    if case["op"] == "norm":
        m = x.mean(1, keepdim=True)
        r = (x.var(1, unbiased=False, keepdim=True) + _EPS).rsqrt()
        z = (x - m) * r * w + b
        y = {"none": lambda: z, "silu": lambda: z * torch.sigmoid(z),
             "gelu": lambda: z * torch.special.ndtr(z)}[case["act"]]()
        return unrows(y), stat(m), stat(r)
    # the gradients with the saved statistics that the call is given
    m = st["mean"].double().reshape(-1, 1)
    r = st["rstd"].double().reshape(-1, 1)
    xh = (x - m) * r
    z = xh * w + b
    if case["act"] == "silu":
        sg = torch.sigmoid(z)
        slope = sg + z * sg * (1.0 - sg)
    elif case["act"] == "gelu":
        slope = torch.special.ndtr(z) + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
    else:
        slope = torch.ones_like(z)
    dz = rows(st["dy"]) * slope
    u = dz * w
    dx = r * (u - u.mean(1, keepdim=True) - xh * (u * xh).mean(1, keepdim=True))
    return unrows(dx), unrows(dz * xh).sum((0, 1)), unrows(dz).sum((0, 1))
