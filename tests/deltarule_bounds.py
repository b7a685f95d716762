"""Reference values of the gated delta rule (float64 on the CPU) and how far float32 and
bfloat16 calls may be off.

Every result is a sum of products; call the root of the sum of its squared terms
its size (o: scale^2 sum q^2 S^2, x: v^2 + sum k^2 S^2, and so on), the largest of
a head's tokens.  Let e be the unit of a rounding: 2^-23 for float32 sums (the
rounding of a product and of its addition), 2^-16 for values kept in two bfloat16
parts, and K = d_qk + 4 * 32 + 64 + T: terms of a sum over d_qk, over a chunk's 32
tokens (in the triangular system, its inverse, the scores and the state), some
single roundings, and one of the state a token (the recurrence itself does not
amplify them: |I - beta k k^T| <= 1 for 0 <= beta |k|^2 <= 2).

Roundings are independent: K of them are sqrt(K) e of the size in the root mean
square.  A triangular system carries what its right side is off by through its
inverse, r the largest row sum of the inverses' magnitudes: (1 + r) sqrt(K) e.
The largest of up to 10^6 values is within eight standard deviations (2 exp(-32)
each).  A bfloat16 result is rounded once more, 2^-8 of itself at most.
"""
import numpy as np
import torch

U = 2.0 ** -24


def sweep(d, lengths, scale):
    """Token-by-token values, float64 torch, with the squared sizes of each (names
    ending in 2).  d: q, k, v, g, beta, do, S0, dS (the last three may be None)."""
    f = {n: None if t is None else t.double().cpu() for n, t in d.items()}
    B, H, T, dv = f["v"].shape
    r = H // f["q"].shape[1]
    q, k = (f[n].repeat_interleave(r, 1) for n in ("q", "k"))
    v, g, beta, do = f["v"], f["g"], f["beta"], f["do"]
    dk = q.shape[-1]
    zero = torch.zeros((B, H, dk, dv), dtype=torch.float64)
    S = zero.clone() if f.get("S0") is None else f["S0"].clone()
    n = torch.tensor([T if lengths is None else min(max(int(lengths[b]), 0), T) for b in range(B)])
    live = torch.arange(T)[None, :] < n[:, None]
    m = live[:, None, :]
    gam = torch.where(m, torch.exp(g), torch.ones(()).double())
    beta = torch.where(m, beta, torch.zeros(()).double())
    z = lambda t: torch.where(m[..., None], t, torch.zeros(()).double())
    q, k, v = z(q), z(k), z(v)
    do = None if do is None else z(do)
    w = dict(k=k, beta=beta, gam=gam)
    left = lambda a, M: (a[:, :, None, :] @ M)[:, :, 0]         # a^T M
    right = lambda M, a: (M @ a[..., None])[..., 0]             # M a
    outer = lambda a, c: a[..., None] * c[:, :, None, :]
    before, x, o, x2, o2 = [], torch.zeros_like(v), torch.zeros_like(v), torch.zeros_like(v), torch.zeros_like(v)
    S2 = S * S
    for t in range(T):
        S = gam[:, :, t, None, None] * S
        before.append(S)          # decayed, before the token's writing
        x[:, :, t] = v[:, :, t] - left(k[:, :, t], S)
        x2[:, :, t] = v[:, :, t] ** 2 + left(k[:, :, t] ** 2, S * S)
        S = S + outer(k[:, :, t], beta[:, :, t, None] * x[:, :, t])
        S2 = torch.maximum(S2, S * S + outer(k[:, :, t] ** 2, beta[:, :, t, None] ** 2 * x2[:, :, t]))
        o[:, :, t] = scale * left(q[:, :, t], S)
        o2[:, :, t] = scale ** 2 * left(q[:, :, t] ** 2, S2)
    w.update(o=o, S=S, o2=o2, S2=S2.amax(2, keepdim=True).expand_as(S))
    if do is None:
        return w
    D = zero.clone() if f.get("dS") is None else f["dS"].clone()
    D2 = D * D
    dq, dkk, dq2, dk2 = (torch.zeros_like(q) for _ in range(4))
    du, du2, db2 = torch.zeros_like(v), torch.zeros_like(v), torch.zeros_like(g)
    dg, dg2 = torch.zeros_like(g), torch.zeros_like(g)
    for t in range(T - 1, -1, -1):
        kt, bt = k[:, :, t], beta[:, :, t, None]
        u, u2 = bt * x[:, :, t], bt ** 2 * x2[:, :, t]
        dq[:, :, t] = scale * right(before[t] + outer(kt, u), do[:, :, t])
        dq2[:, :, t] = scale ** 2 * right(S2, do[:, :, t] ** 2)
        D = D + scale * outer(q[:, :, t], do[:, :, t])
        D2 = torch.maximum(D2, D * D + scale ** 2 * outer(q[:, :, t] ** 2, do[:, :, t] ** 2))
        du[:, :, t], du2[:, :, t] = left(kt, D), left(kt ** 2, D2)
        dvt = bt * du[:, :, t]
        dkk[:, :, t] = right(D, u) - right(before[t], dvt)
        dk2[:, :, t] = right(D2, u2) + right(S2, bt ** 2 * du2[:, :, t])
        db2[:, :, t] = (du2[:, :, t] * x2[:, :, t]).sum(-1)
        D = D - outer(kt, dvt)
        dg[:, :, t] = (D * before[t]).sum((-1, -2))
        # the same through up to 128 tokens' q.dq + k.dk - 2 beta dbeta
        dg2[:, :, t] = (D2 * S2).sum((-1, -2))
        D = gam[:, :, t, None, None] * D
    dg2 = dg2 + 128 * ((q ** 2 * dq2).sum(-1) + (k ** 2 * dk2).sum(-1) + 4 * beta ** 2 * db2).amax(2, keepdim=True)
    group = lambda t: t.reshape(B, H // r, r, T, dk).sum(2)
    w.update(dv=beta[..., None] * du, dv2=beta[..., None] ** 2 * du2, dbeta=(du * x).sum(-1) * m, dbeta2=db2,
             dg=dg * m, dg2=dg2, dS0=D, dS02=D2.amax(2, keepdim=True).expand_as(D), dq=group(dq), dq2=group(dq2),
             dk=group(dkk), dk2=group(dk2), T=T)
    return w


def _row_sums(w):
    """Largest row sum of |inverse| over all 32-token chunks of each head."""
    k, beta, gam = w["k"], w["beta"], w["gam"]
    B, H, T, _ = k.shape
    pad = -T % 32
    k = torch.nn.functional.pad(k, (0, 0, 0, pad)).reshape(B, H, -1, 32, k.shape[-1])
    beta = torch.nn.functional.pad(beta, (0, pad)).reshape(B, H, -1, 1, 32)
    G = torch.nn.functional.pad(gam, (0, pad), value=1.0).reshape(B, H, -1, 32).clamp(min=1e-300).log().cumsum(-1)
    M = torch.exp((G[..., :, None] - G[..., None, :]).clamp(max=0.0))
    A = torch.tril(M * (k @ k.transpose(-1, -2)), -1) * beta
    inv = torch.linalg.inv(torch.eye(32, dtype=torch.float64) + A)
    return torch.maximum(inv.abs().sum(-1), inv.transpose(-1, -2).abs().sum(-1)).amax((-1, -2))  # [B, H]


def check(w, got, io, what):
    """Results ``got`` (a dict by name) against the sweep w of the same call."""
    T = w["beta"].shape[2]
    root = (w["k"].shape[-1] + 4 * 32 + 64 + T) ** 0.5
    rows = _row_sums(w)                                   # [B, H]
    for name, x in got.items():
        ref, size2 = w[name], w[name + "2"]
        x = x.detach().double().cpu()
        assert x.shape == ref.shape and bool(torch.isfinite(x).all()), f"{what} {name}"
        state = name in ("S", "dS0")
        e = 2.0 ** -16 if io == "bf16" and not state else 2.0 ** -23
        r = rows
        if ref.shape[1] != rows.shape[1]:                 # shared heads: the worst of a group
            r = rows.reshape(rows.shape[0], ref.shape[1], -1).amax(2)
        size2 = size2 if state else size2.amax(2, keepdim=True)
        one = (1 + r).reshape(r.shape + (1,) * (ref.dim() - 2)) * root * e * size2.sqrt().expand_as(ref)
        rounded = 2.0 ** -8 if io == "bf16" and name in ("o", "dq", "dk", "dv") else U
        err = (x - ref).abs()
        part = float((err / (8 * one + rounded * ref.abs() + 1e-30)).max())
        rms = lambda t: float((t ** 2).mean().sqrt())
        rel = rms(err) / (rms(one) + rounded * rms(ref) + 1e-30)
        print(f"[delta] {what} {name}: largest {part:.4f} of the bound, rms {rel:.4f} of it, "
              f"{rms(err) / max(rms(ref), 1e-30):.2e} of the values", flush=True)
        assert part <= 1.0, (what, name, part)
        assert rel <= 1.0, (what, name, rel)
