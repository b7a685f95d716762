"""Workloads of the gated delta rule and of the norm and rotation of queries and
keys: their inputs, their plain forms in elementary torch operations, their
exact values and the work that each cannot do without.

Gated delta rule (state S [d_k, d_v] of each head; a log decay g_t <= 0 and a
writing strength beta_t for each token):

    S_t = e^{g_t} (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,
    o_t = scale * S_t^T q_t

as whole sequences (``prefill``), a single token (``step``) and the gradients of
a sequence (``backward``).  Heads of values may share heads of queries and keys.

Norm and rotation of queries and keys (``qk``, gradients ``qk_grad``): each
head's row is divided by its length (``l2``) or its root mean square (``rms``),
scaled by a weight, and its first channels are rotated by the token's position,
in pairs of halves or of neighbours.
"""
import math

import torch

own = False   # True: the library's kernels; False: the plain forms below

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_EPS = 1e-6


# ---------------------------------------------------------------- cases

def _seq(name, op, B, Hk, H, T, dk, dv, io, ragged=False, token_major=False, state=False):
    c = {"op": op, "B": B, "Hk": Hk, "H": H, "T": T, "dk": dk, "dv": dv, "io": io, "ragged": ragged,
         "token_major": token_major, "state": state}
    return {"name": name, **c} if name else c


def _step(name, B, Hk, H, dk, dv, io):
    c = {"op": "step", "B": B, "Hk": Hk, "H": H, "dk": dk, "dv": dv, "io": io}
    return {"name": name, **c} if name else c


def _qk(name, op, B, T, H, Hk, d, io, norm, rot=0, layout="half", far=0, factor=1.0):
    c = {"op": op, "B": B, "T": T, "H": H, "Hk": Hk, "d": d, "io": io, "norm": norm, "rot": rot,
         "layout": layout, "far": far, "factor": factor}
    return {"name": name, **c} if name else c


def listed():
    return [
        # a short prompt continued from a state, float32: latency counts
        _seq("prefill_short_f32", "prefill", 1, 4, 4, 37, 64, 64, "f32", state=True),
        # a padded batch of prompts read straight out of a fused projection
        # (token-major rows), two value heads to a key head, lengths from the full
        # 2000 down to an empty one
        _seq("prefill_padded_bf16", "prefill", 6, 8, 16, 2000, 128, 128, "bf16", ragged=True,
             token_major=True, state=True),
        # the sequence shape of the library's own 7B-layer prefill workload
        _seq("prefill_7b_bf16", "prefill", 8, 8, 8, 4096, 256, 512, "bf16"),
        # one long document: few heads in flight, many chunks in a row
        _seq("prefill_long_bf16", "prefill", 1, 8, 8, 32768, 128, 128, "bf16", state=True),
        # single tokens of a small and of the library's decode batch
        _step("step_small_bf16", 3, 8, 8, 64, 64, "bf16"),
        _step("step_batch_bf16", 256, 8, 8, 256, 512, "bf16"),
        # gradients at the library's float32 training shape, carried state included
        _seq("backward_small_f32", "backward", 4, 4, 4, 1024, 64, 64, "f32", state=True),
        # a training step's gradients of one layer of 16 heads of 128
        _seq("backward_layer_bf16", "backward", 4, 16, 16, 4096, 128, 128, "bf16", token_major=True),
        # queries and keys of unit length, as they go into the delta rule's prefill
        _qk("qk_unit_bf16", "qk", 4, 4096, 16, 16, 128, "bf16", "l2"),
        # a decode batch: one row a head, rotated in part, each sequence at its own position
        _qk("qk_decode_bf16", "qk", 64, 1, 8, 2, 256, "bf16", "rms", rot=64, far=100000),
        # neighbouring pairs, channels that fill no wavefront, an odd number of tokens
        _qk("qk_pairs_f32", "qk", 3, 1301, 10, 5, 96, "f32", "rms", rot=72, layout="pairs"),
        # a training step's gradients, shared key heads, positions stretched to a long context
        _qk("qk_grad_bf16", "qk_grad", 4, 4096, 16, 4, 128, "bf16", "rms", rot=128, far=400000, factor=8.0),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "step", "backward", "backward", "qk", "qk_grad"])
    io = rng.choice(["f32", "bf16", "bf16"])
    if op in ("prefill", "backward"):
        dk = 16 * _logint(rng, 1, 16)
        dv = 16 * _logint(rng, 1, 32)
        B, Hk, r = _logint(rng, 1, 16), _logint(rng, 1, 16), rng.choice([1, 1, 2, 3])
        H = Hk * r
        # tokens so that the case's products and rows stay below the largest listed ones'
        cap = min(2.5e10 / (dk * dv), 3e8 / (2 * dk + 2 * dv)) if op == "prefill" \
            else min(4e9 / (dk * dv), 1.8e8 / (4 * dk + 3 * dv))
        cap /= B * H * (8 if io == "f32" else 1)
        T = _logint(rng, 1, max(1, min(16384, int(cap))))
        return _seq(None, op, B, Hk, H, T, dk, dv, io, ragged=B > 1 and rng.random() < 0.5,
                    token_major=rng.random() < 0.5, state=rng.random() < 0.5)
    if op == "step":
        dk = 16 * _logint(rng, 1, 16)
        dv = 16 * _logint(rng, 1, 32)
        Hk, r = _logint(rng, 1, 16), rng.choice([1, 1, 2, 3])
        H = Hk * r
        B = _logint(rng, 1, max(1, min(512, int(2.6e8 / (H * dk * dv)))))
        return _step(None, B, Hk, H, dk, dv, io)
    d = rng.choice([_logint(rng, 2, 512), 16 * _logint(rng, 1, 32), 16 * _logint(rng, 1, 32)])
    Hk, r = _logint(rng, 1, 16), rng.choice([1, 1, 2, 4])
    B = _logint(rng, 1, 64)
    T = _logint(rng, 1, max(1, min(16384, int(3e7 / (B * Hk * (r + 1) * d)))))
    rot = 0 if rng.random() < 0.25 else 2 * _logint(rng, 1, d // 2)
    norm = rng.choice(["rms", "l2"]) if rot == 0 else rng.choice(["rms", "l2", "none"])
    return _qk(None, op, B, T, Hk * r, Hk, d, io, norm, rot=rot, layout=rng.choice(["half", "pairs"]),
               far=rng.choice([0, 5000, 1000000]), factor=rng.choice([1.0, 4.0]))


# ---------------------------------------------------------------- inputs

def _lengths(case):
    """Tokens of each sequence of a padded batch: the first is full, the last empty."""
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return [T] * B
    return [T * (B - 1 - b) // (B - 1) for b in range(B)]


def _gen(seed, dev="cuda"):
    g = torch.Generator(device=dev)
    g.manual_seed(0x5DE1 + 7919 * int(seed))
    return g


def _rand(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device=g.device) * std


def _unit(x):
    """Rows as they come out of a projection, SiLU and the division by their length."""
    x = x / (1.0 + torch.exp(-x))
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) + _EPS)


def _heads(case, make, H, d):
    """A [B, H, T, d] tensor, dense or as a view of token-major [B, T, H, d] rows."""
    B, T = case["B"], case["T"]
    if case["token_major"]:
        return make((B, T, H, d)).transpose(1, 2)
    return make((B, H, T, d))


def _gates(g, H, rows):
    """log decays g = -a softplus(.), a from a memory of a few tokens to one of
    hundreds over the heads, and strengths beta = sigmoid(.); heads last."""
    a = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32, device="cuda")
    z = _rand(g, rows + (H,))
    decay = -a * torch.log1p(torch.exp(z))
    return decay.float(), (1.0 / (1.0 + torch.exp(-_rand(g, rows + (H,))))).float()


def _frequencies(rot, factor):
    """Rotations per position in radians, base 10000: fast pairs as they are, slow
    ones (fewer than one turn over 4096 positions) slowed by the factor, a ramp between."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    turns = 4096.0 * f / (2.0 * math.pi)
    keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
    return (f * keep + f / factor * (1.0 - keep)).float().cuda()


def prepare(case, seed):
    g = _gen(seed)
    dt = _DT[case["io"]]
    op = case["op"]
    st = {"case": case}
    if op in ("qk", "qk_grad"):
        B, T, H, Hk, d, rot = (case[x] for x in ("B", "T", "H", "Hk", "d", "rot"))
        # queries and keys as views of a fused projection's rows
        rows = _rand(g, (B, T, H + Hk, d)).to(dt)
        st["q"], st["k"] = rows[:, :, :H].transpose(1, 2), rows[:, :, H:].transpose(1, 2)
        st["wq"] = st["wk"] = None
        if case["norm"] == "rms":
            st["wq"], st["wk"] = 1.0 + 0.2 * _rand(g, (d,)), 1.0 + 0.2 * _rand(g, (d,))
        st["freq"] = _frequencies(rot, case["factor"]) if rot else None
        start = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device="cuda", dtype=torch.int32)
        st["pos"] = (start + torch.arange(T, device="cuda", dtype=torch.int32)) if rot else None
        st["amp"] = 1.0 + 0.1 * math.log(case["factor"])
        if op == "qk_grad":
            st["dyq"] = _rand(g, (B, H, T, d)).to(dt)
            st["dyk"] = _rand(g, (B, Hk, T, d)).to(dt)
        return st
    B, Hk, H, dk, dv = (case[x] for x in ("B", "Hk", "H", "dk", "dv"))
    st["scale"] = dk ** -0.5
    if op == "step":
        st["q"], st["k"] = _unit(_rand(g, (B, Hk, dk))).to(dt), _unit(_rand(g, (B, Hk, dk))).to(dt)
        st["v"] = _rand(g, (B, H, dv)).to(dt)
        st["g"], st["beta"] = _gates(g, H, (B,))
        st["S"] = _rand(g, (B, H, dk, dv), 0.1)
        st["S_out"] = torch.empty_like(st["S"])
        return st
    unit = lambda s: _unit(_rand(g, s)).to(dt)
    wide = lambda s: _rand(g, s).to(dt)
    st["q"], st["k"] = _heads(case, unit, Hk, dk), _heads(case, unit, Hk, dk)
    st["v"] = _heads(case, wide, H, dv)
    # gates come out of a projection too: [B, T, H], seen as [B, H, T]
    decay, beta = _gates(g, H, (B, case["T"]))
    st["g"], st["beta"] = decay.transpose(1, 2), beta.transpose(1, 2)
    if not case["token_major"]:
        st["g"], st["beta"] = st["g"].contiguous(), st["beta"].contiguous()
    st["S0"] = _rand(g, (B, H, dk, dv), 0.1) if case["state"] else None
    st["lengths"] = (torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
                     if case["ragged"] else None)
    if op == "backward":
        st["do"] = _heads(case, wide, H, dv)
        st["dS"] = _rand(g, (B, H, dk, dv), 0.1) if case["state"] else None
    return st


# ---------------------------------------------------------------- plain forms

_CHUNK = 64


def _rows(st, *names):
    """Float32 copies [B, H, N, C, .] in chunks of C tokens, one row for each value
    head; rows that are no tokens are zeros."""
    T = st["v"].shape[2]
    H = st["v"].shape[1]
    pad = -T % _CHUNK
    L = st["lengths"]
    mask = None if L is None else (torch.arange(T, device="cuda")[None, :] < L[:, None])[:, None, :, None]
    out = []
    for n in names:
        x = st[n].float()
        if x.dim() == 3:
            x = x[..., None]
        if mask is not None:
            x = torch.where(mask, x, torch.zeros((), device="cuda"))
        if x.shape[1] != H:
            x = x.repeat_interleave(H // x.shape[1], 1)
        if pad:
            x = torch.cat([x, torch.zeros(x.shape[:2] + (pad, x.shape[3]), device="cuda")], 2)
        out.append(x.reshape(x.shape[0], H, -1, _CHUNK, x.shape[3]).contiguous())
    return out


def _tr(x):
    return x.transpose(-1, -2).contiguous()


def _inside(q, k, g, beta):
    """What a chunk computes without the state: the decays e^{G_i}, e^{G_L - G_j}
    and M_ij = e^{G_i - G_j} (j <= i), the products M q k^T and M k k^T (j < i), and
    the inverse of I + (M k k^T) beta, row by row."""
    G = torch.cumsum(g.double(), -2)
    C = G.shape[-2]
    M = torch.exp((G - G.transpose(-1, -2)).clamp(max=0.0)).float()
    low = torch.tril(torch.ones((C, C), device="cuda"))
    strict = low - torch.eye(C, device="cuda")
    kt = _tr(k)
    P = torch.matmul(q, kt) * M * low
    N = torch.matmul(k, kt) * M * strict
    A = N * beta.transpose(-1, -2)
    inv = torch.eye(C, device="cuda").expand(A.shape).clone()
    for i in range(1, C):
        inv[..., i, :i] = -torch.matmul(A[..., i:i + 1, :i].contiguous(), inv[..., :i, :i].contiguous())[..., 0, :]
    return M, P, N, inv, torch.exp(G).float(), torch.exp(G[..., -1:, :] - G).float()


def _sweep(st, q, k, v, g, beta, keep):
    """The chunks in order: outputs (None without q) and the state before each
    chunk (with keep) and after the last one."""
    B, H, N, C, dk = k.shape
    dv = v.shape[-1]
    M, P, _, inv, fade, rest = _inside(q, k, g, beta)
    W = torch.matmul(inv, fade * k)
    V = torch.matmul(inv, v)
    S = st["S0"] if st["S0"] is not None else torch.zeros((B, H, dk, dv), device="cuda")
    o = torch.empty((B, H, N, C, dv), device="cuda")
    X = torch.empty((B, H, N, C, dv), device="cuda")
    states = []
    for c in range(N):
        if keep:
            states.append(S)
        x = V[:, :, c] - torch.matmul(W[:, :, c], S)
        u = beta[:, :, c] * x
        X[:, :, c] = x
        o[:, :, c] = (torch.matmul(fade[:, :, c] * q[:, :, c], S) + torch.matmul(P[:, :, c], u)) * st["scale"]
        S = fade[:, :, c, -1:] * S + torch.matmul(_tr(rest[:, :, c] * k[:, :, c]), u)
    return o, X, states, S


def _unchunk(x, T):
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])[:, :, :T]


def _plain_prefill(st):
    q, k, v, g, beta = _rows(st, "q", "k", "v", "g", "beta")
    o, _, _, S = _sweep(st, q, k, v, g, beta, False)
    return _unchunk(o, st["v"].shape[2]).to(st["q"].dtype), S


def _plain_step(st):
    r = st["v"].shape[1] // st["q"].shape[1]
    q, k = (st[n].float().repeat_interleave(r, 1) for n in ("q", "k"))
    S = torch.exp(st["g"])[..., None, None] * st["S"]
    x = st["v"].float() - (k[..., None] * S).sum(-2)
    S = S + (st["beta"][..., None] * k)[..., None] * x[..., None, :]
    o = (q[..., None] * S).sum(-2) * st["scale"]
    return o.to(st["q"].dtype), S


def _plain_backward(st):
    q, k, v, g, beta, do = _rows(st, "q", "k", "v", "g", "beta", "do")
    B, H, N, C, dk = k.shape
    dv, s, T = v.shape[-1], st["scale"], st["v"].shape[2]
    M, P, NN, inv, fade, rest = _inside(q, k, g, beta)
    _, X, states, S = _sweep(st, q, k, v, g, beta, True)
    states.append(S)
    S = torch.stack(states, 2)                     # [B, H, N + 1, dk, dv]
    # the state's gradient, chunk by chunk from the last one
    D = st["dS"] if st["dS"] is not None else torch.zeros((B, H, dk, dv), device="cuda")
    back, Ds, dX, dU = _tr(inv), [], torch.empty_like(X), torch.empty_like(X)
    for c in range(N - 1, -1, -1):
        Ds.append(D)
        u = torch.matmul(_tr(P[:, :, c]), do[:, :, c]) * s + torch.matmul(rest[:, :, c] * k[:, :, c], D)
        x = torch.matmul(back[:, :, c], beta[:, :, c] * u)
        dX[:, :, c] = x
        dU[:, :, c] = u - torch.matmul(_tr(NN[:, :, c]), x)
        D = fade[:, :, c, -1:] * D + torch.matmul(_tr(fade[:, :, c] * q[:, :, c]), do[:, :, c]) * s \
            - torch.matmul(_tr(fade[:, :, c] * k[:, :, c]), x)
    end = torch.stack(Ds[::-1], 2)
    low = torch.tril(torch.ones((C, C), device="cuda"))
    U = beta * X
    E1 = torch.matmul(do, _tr(U)) * M * low
    E2 = torch.matmul(dX, _tr(U)) * M * (low - torch.eye(C, device="cuda"))
    dq = (fade * torch.matmul(do, _tr(S[:, :, :-1])) + torch.matmul(E1, k)) * s
    dkk = rest * torch.matmul(U, _tr(end)) - fade * torch.matmul(dX, _tr(S[:, :, :-1])) \
        + torch.matmul(_tr(E1), q) * s - torch.matmul(E2 + _tr(E2), k)
    dbeta = (dU * X).sum(-1)
    dG = (q * dq).sum(-1) - (dX * v).sum(-1)
    tail = (end * S[:, :, 1:]).sum((-1, -2))
    dg = torch.flip(torch.cumsum(torch.flip(dG, (-1,)), -1), (-1,)) + tail[..., None]
    if st["lengths"] is not None:
        t = torch.arange(N * C, device="cuda").reshape(1, 1, N, C)
        dg = torch.where(t < st["lengths"].reshape(-1, 1, 1, 1), dg, torch.zeros((), device="cuda"))
    Hk = st["q"].shape[1]
    heads = lambda x: _unchunk(x, T).reshape(B, Hk, H // Hk, T, -1).sum(2)
    dt = st["q"].dtype
    out = (heads(dq).to(dt), heads(dkk).to(dt), _unchunk(dX, T).to(dt), dg.reshape(B, H, -1)[:, :, :T],
           dbeta.reshape(B, H, -1)[:, :, :T])
    return out + (D,) if st["dS"] is not None else out


def _inv_norm(x, norm):
    if norm == "none":
        return torch.ones_like(x[..., :1])
    sq = (x * x).sum(-1, keepdim=True)
    return torch.rsqrt((sq if norm == "l2" else sq / x.shape[-1]) + _EPS)


def _angles(st):
    """cos and sin [B, 1, T, rot / 2] times the amplitude; the angles in 64 bits."""
    a = st["pos"].double()[:, None, :, None] * st["freq"].double()
    return (torch.cos(a) * st["amp"]).float(), (torch.sin(a) * st["amp"]).float()


def _turn(x, c, s, layout):
    """The first channels' pairs turned by (c, s)."""
    r = 2 * c.shape[-1]
    h = r // 2
    y = x.clone()
    a, b = (x[..., :h], x[..., h:r]) if layout == "half" else (x[..., 0:r:2], x[..., 1:r:2])
    u, v = a * c - b * s, b * c + a * s
    if layout == "half":
        y[..., :h], y[..., h:r] = u, v
    else:
        y[..., 0:r:2], y[..., 1:r:2] = u, v
    return y


def _plain_qk(st):
    case = st["case"]
    cs = _angles(st) if case["rot"] else None
    out = []
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        y = x.float()
        y = y * _inv_norm(y, case["norm"])
        if w is not None:
            y = y * w
        if cs:
            y = _turn(y, *cs, case["layout"])
        out.append(y.to(x.dtype))
    return tuple(out)


def _plain_qk_grad(st):
    case = st["case"]
    cs = _angles(st) if case["rot"] else None
    dx, dw = [], []
    for x, w, dy in ((st["q"], st["wq"], st["dyq"]), (st["k"], st["wk"], st["dyk"])):
        d = dy.float()
        if cs:
            d = _turn(d, cs[0], -cs[1], case["layout"])
        x32 = x.float()
        r = _inv_norm(x32, case["norm"])
        if w is not None:
            dw.append((d * x32 * r).sum((0, 1, 2)))
            d = d * w
        if case["norm"] != "none":
            n = 1 if case["norm"] == "l2" else x.shape[-1]
            d = r * d - x32 * (r * r * r * (d * x32).sum(-1, keepdim=True) / n)
        dx.append(d.to(x.dtype))
    return tuple(dx + dw)


_PLAIN = {"prefill": _plain_prefill, "step": _plain_step, "backward": _plain_backward,
          "qk": _plain_qk, "qk_grad": _plain_qk_grad}


# ---------------------------------------------------------------- one pass

def run(st):
    c = st["case"]
    op = c["op"]
    if not own:
        return _PLAIN[op](st)
    from xlstm_mlstm_matrix_amd import binding as B
    if op == "prefill":
        return B.deltarule_fwd(st["q"], st["k"], st["v"], st["g"], st["beta"], st["S0"],
                               lengths=st["lengths"], scale=st["scale"])
    if op == "step":
        return B.deltarule_step(st["q"], st["k"], st["v"], st["g"], st["beta"], st["S"], scale=st["scale"],
                                S_out=st["S_out"])
    if op == "backward":
        return B.deltarule_bwd(st["q"], st["k"], st["v"], st["g"], st["beta"], st["do"], st["S0"], st["dS"],
                               lengths=st["lengths"], scale=st["scale"], state_grad=st["dS"] is not None)
    kw = dict(norm=c["norm"], eps=_EPS, inv_freq=st["freq"], positions=st["pos"], layout=c["layout"],
              amplitude=st["amp"])
    if op == "qk":
        return B.qknorm_fwd(st["q"], st["k"], st["wq"], st["wk"], **kw)
    dq, dk, dwq, dwk = B.qknorm_bwd(st["q"], st["k"], st["dyq"], st["dyk"], st["wq"], st["wk"], **kw)
    return (dq, dk) if st["wq"] is None else (dq, dk, dwq, dwk)


# ---------------------------------------------------------------- work

def work(case):
    """Each input read once, each output written once; multiply-adds of the recurrent form."""
    op = case["op"]
    e = 4 if case["io"] == "f32" else 2
    if op in ("qk", "qk_grad"):
        n = case["B"] * case["T"] * (case["H"] + case["Hk"]) * case["d"]
        pos = 4 * case["B"] * case["T"] if case["rot"] else 0
        if op == "qk":
            return {"bytes": 2 * n * e + pos, "flops": 8 * n}
        return {"bytes": 3 * n * e + pos, "flops": 16 * n}
    B, Hk, H, dk, dv = (case[x] for x in ("B", "Hk", "H", "dk", "dv"))
    if op == "step":
        return {"bytes": B * H * (8 * dk * dv + e * 2 * dv + 8) + e * B * Hk * 2 * dk, "flops": B * H * 8 * dk * dv}
    rows = sum(_lengths(case))
    all_rows = B * case["T"]
    state = B * H * dk * dv * 4
    if op == "prefill":
        # q, k, v and the gates of the real tokens, o of all rows; the state in and out
        b = e * (rows * (2 * Hk * dk + H * dv) + all_rows * H * dv) + 8 * rows * H
        return {"bytes": b + state * (2 if case["state"] else 1), "flops": rows * H * 7 * dk * dv}
    b = e * (rows * (2 * Hk * dk + 2 * H * dv) + all_rows * (2 * Hk * dk + H * dv)) + 8 * (rows + all_rows) * H
    return {"bytes": b + state * (3 if case["state"] else 0), "flops": rows * H * 18 * dk * dv}


# ---------------------------------------------------------------- exact values

def exact(case, seed):
    """The recurrences token by token, and norm and rotation from their definitions, in float64."""
    op = case["op"]
    st = prepare(case, seed)
    if op == "qk":
        return _exact_qk(case, st)
    if op == "qk_grad":
        return _exact_qk_grad(case, st)
    if op == "step":
        H = case["H"]
        own_head = torch.arange(H, device="cuda") // (H // case["Hk"])
        q, k = st["q"].double()[:, own_head], st["k"].double()[:, own_head]
        v, S = st["v"].double(), st["S"].double()
        gam, beta = torch.exp(st["g"].double()), st["beta"].double()
        kS = (k.unsqueeze(-2) @ S).squeeze(-2)
        # e^g (S - beta k (k^T S)) + beta k v^T
        S = gam[..., None, None] * (S - (beta[..., None] * k)[..., None] * kS[..., None, :]) \
            + (beta[..., None] * k)[..., None] * v[..., None, :]
        return (q.unsqueeze(-2) @ S).squeeze(-2) * st["scale"], S
    return _exact_sequence(case, st)


def _exact_sequence(case, st):
    B, Hk, H, T, dk, dv = (case[x] for x in ("B", "Hk", "H", "T", "dk", "dv"))
    # each token reads and writes the whole state a few times, in float64
    if T * (2e-4 + B * H * dk * dv * 64 / 1.5e12) * (1 if case["op"] == "prefill" else 3) > 20.0:
        return None
    s = st["scale"]
    L = _lengths(case)
    # sequences in order of their length, so those still running are the first ones
    order = sorted(range(B), key=lambda b: -L[b])
    perm = torch.tensor(order, device="cuda")
    live = [sum(1 for b in range(B) if L[b] > t) for t in range(T)]
    own_head = torch.arange(H, device="cuda") // (H // Hk)
    z = lambda *d: torch.zeros((T, B, H) + d, dtype=torch.float64, device="cuda")

    def tok(n):   # [T, B, H, ...], a copy of the shared rows for each head
        x = st[n].double()[perm]
        if x.shape[1] != H:
            x = x[:, own_head]
        return x.permute((2, 0, 1) + tuple(range(3, x.dim()))).contiguous()

    start = lambda n: (torch.zeros((B, H, dk, dv), dtype=torch.float64, device="cuda")
                       if st[n] is None else st[n].double()[perm])
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(B, device="cuda")

    def back(x):
        return x.permute((1, 2, 0) + tuple(range(3, x.dim())))[inv]

    q, k, v, beta = tok("q"), tok("k"), tok("v"), tok("beta")
    gam = torch.exp(tok("g"))

    def forward(S, t, n):
        """One token: decay, the value that is missing, its writing."""
        S.mul_(gam[t, :n, :, None, None])
        x = v[t, :n] - (k[t, :n, :, None, :] @ S)[:, :, 0]
        S.addcmul_(k[t, :n, :, :, None], (beta[t, :n, :, None] * x)[:, :, None, :])
        return x

    S = start("S0")
    if case["op"] == "prefill":
        o = z(dv)
        for t in range(T):
            n = live[t]
            if n == 0:
                break
            forward(S[:n], t, n)
            o[t, :n] = (q[t, :n, :, None, :] @ S[:n])[:, :, 0] * s
        return back(o), S[inv]
    do = tok("do")
    dq, dkk, x = z(dk), z(dk), z(dv)
    for t in range(T):
        n = live[t]
        if n == 0:
            break
        x[t, :n] = forward(S[:n], t, n)
        dq[t, :n] = (S[:n] @ do[t, :n, :, :, None])[..., 0] * s
    D = start("dS")
    last = (D * S).sum((-1, -2))
    dvv, dbeta = z(dv), z()
    for t in range(T - 1, -1, -1):
        n = live[t]
        if n == 0:
            continue
        Dn = D[:n]
        Dn.addcmul_(q[t, :n, :, :, None], do[t, :n, :, None, :], value=s)
        dkk[t, :n] = (Dn @ (beta[t, :n, :, None] * x[t, :n])[..., None])[..., 0]
        du = (k[t, :n, :, None, :] @ Dn)[:, :, 0]
        dbeta[t, :n] = (du * x[t, :n]).sum(-1)
        dvv[t, :n] = beta[t, :n, :, None] * du
        Dn.addcmul_(k[t, :n, :, :, None], dvv[t, :n, :, None, :], value=-1.0)
        Dn.mul_(gam[t, :n, :, None, None])
    # the part of dk that reads the decayed state before its token
    S = start("S0")
    for t in range(T):
        n = live[t]
        if n == 0:
            break
        S[:n].mul_(gam[t, :n, :, None, None])
        dkk[t, :n] -= (S[:n] @ dvv[t, :n, :, :, None])[..., 0]
        S[:n].addcmul_(k[t, :n, :, :, None], (beta[t, :n, :, None] * x[t, :n])[:, :, None, :])
    # a decay scales every later output and the final state, less what v adds
    dG = (q * dq).sum(-1) - (dvv * v).sum(-1)
    for b in range(B):
        if L[order[b]] < T:
            dG[L[order[b]]:, b] = 0.0
    dg = torch.flip(torch.cumsum(torch.flip(dG, (0,)), 0), (0,)) + last[None]
    for b in range(B):
        dg[L[order[b]]:, b] = 0.0
    shared = lambda x: back(x).reshape(B, Hk, H // Hk, T, -1).sum(2)
    out = (shared(dq), shared(dkk), back(dvv), back(dg), back(dbeta))
    return out + (D[inv],) if st["dS"] is not None else out


def _exact_norms(case, x):
    """1 / length or 1 / root mean square of each row [B, T, heads, d]."""
    if case["norm"] == "none":
        return torch.ones(x.shape[:-1], dtype=torch.float64, device="cuda")
    sq = torch.linalg.vector_norm(x, dim=-1) ** 2
    return 1.0 / torch.sqrt((sq if case["norm"] == "l2" else sq / case["d"]) + _EPS)


def _exact_rotation(case, st, x, sign):
    """Pairs as complex numbers times amplitude e^{i angle}, rows [B, T, heads, d]."""
    rot = case["rot"]
    if rot == 0:
        return x
    angle = torch.outer(st["pos"].double().reshape(-1), st["freq"].double()).reshape(case["B"], case["T"], 1, rot // 2)
    turn = torch.polar(torch.full_like(angle, st["amp"]), sign * angle)
    pairs = (x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2) if case["layout"] == "half"
             else x[..., :rot].unflatten(-1, (rot // 2, 2)))
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    y = (y.transpose(-1, -2) if case["layout"] == "half" else y).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _exact_qk(case, st):
    out = []
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        x = x.double().transpose(1, 2)
        y = x * _exact_norms(case, x)[..., None]
        y = y if w is None else y * w.double()
        out.append(_exact_rotation(case, st, y, 1.0).transpose(1, 2))
    return tuple(out)


def _exact_qk_grad(case, st):
    dx, dw = [], []
    for x, w, dy in ((st["q"], st["wq"], st["dyq"]), (st["k"], st["wk"], st["dyk"])):
        x, dz = x.double().transpose(1, 2), _exact_rotation(case, st, dy.double().transpose(1, 2), -1.0)
        r = _exact_norms(case, x)[..., None]
        unit = x * r
        if w is not None:
            dw.append(torch.einsum("bthd,bthd->d", dz, unit))
            dz = dz * w.double()
        if case["norm"] != "none":
            n = 1.0 if case["norm"] == "l2" else float(case["d"])
            dz = r * (dz - unit * ((dz * unit).sum(-1, keepdim=True) / n))
        else:
            dz = dz * r
        dx.append(dz.transpose(1, 2))
    return tuple(dx + dw)
