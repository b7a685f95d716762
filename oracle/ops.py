"""float64 oracle of linear attention with a decay for each head, of the gated
delta rule, of group norm with an activation and of the norm and rotation of
queries and keys, written token by token and row by row from the formulas (numpy;
shares nothing with the HIP kernels).

Linear attention, g = log decay of a head, s = scale:

    S_t = e^g S_{t-1} + k_t v_t^T,    o_t = s q_t^T S_t,

and its gradients with D_t = dL/dS_t:

    D_t = e^g D_{t+1} + s q_t do_t^T  (from dL/dS_T at the last token),
    dq_t = s S_t do_t,  dk_t = D_t v_t,  dv_t = D_t^T k_t,  dS_0 = e^g D_0.
"""
import math

import numpy as np


def _np(t):
    return np.asarray(t.detach().double().cpu().numpy() if hasattr(t, "detach") else t, dtype=np.float64)


def linattn_forward(q, k, v, g, S0=None, lengths=None, scale=1.0):
    """(o [B,H,T,dv], S_T [B,H,dk,dv]); rows behind a sequence's length are zero."""
    q, k, v, g = _np(q), _np(k), _np(v), _np(g)
    B, H, T, dk = q.shape
    o = np.zeros((B, H, T, v.shape[-1]))
    S = np.zeros((B, H, dk, v.shape[-1])) if S0 is None else _np(S0).copy()
    gam = np.exp(g)[:, None, None]
    for b in range(B):
        n = T if lengths is None else min(max(int(lengths[b]), 0), T)
        for t in range(n):
            S[b] = gam * S[b] + k[b, :, t, :, None] * v[b, :, t, None, :]
            o[b, :, t] = scale * np.einsum("hk,hkv->hv", q[b, :, t], S[b])
    return o, S


def linattn_backward(q, k, v, g, do, S0=None, dS_T=None, lengths=None, scale=1.0):
    """(dq, dk, dv, dS0)."""
    q, k, v, g, do = _np(q), _np(k), _np(v), _np(g), _np(do)
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    gq, gk, gv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    S = np.zeros((B, H, dk, dv)) if S0 is None else _np(S0).copy()
    D = np.zeros((B, H, dk, dv)) if dS_T is None else _np(dS_T).copy()
    gam = np.exp(g)[:, None, None]
    for b in range(B):
        n = T if lengths is None else min(max(int(lengths[b]), 0), T)
        for t in range(n):
            S[b] = gam * S[b] + k[b, :, t, :, None] * v[b, :, t, None, :]
            gq[b, :, t] = scale * np.einsum("hkv,hv->hk", S[b], do[b, :, t])
        for t in range(n - 1, -1, -1):
            D[b] = D[b] + scale * q[b, :, t, :, None] * do[b, :, t, None, :]
            gk[b, :, t] = np.einsum("hkv,hv->hk", D[b], v[b, :, t])
            gv[b, :, t] = np.einsum("hkv,hk->hv", D[b], k[b, :, t])
            D[b] = gam * D[b]
    return gq, gk, gv, D


def _tokens(lengths, b, T):
    return T if lengths is None else min(max(int(lengths[b]), 0), T)


def deltarule_forward(q, k, v, g, beta, S0=None, lengths=None, scale=1.0):
    """The gated delta rule: S_t = e^{g_t} (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,
    o_t = s q_t^T S_t.  (o [B,H,T,dv], S_T [B,H,dk,dv]); q, k [B,Hk,T,dk]."""
    q, k, v, g, beta = _np(q), _np(k), _np(v), _np(g), _np(beta)
    B, H, T, dv = v.shape
    q, k = (np.repeat(x, H // x.shape[1], 1) for x in (q, k))
    dk = k.shape[-1]
    o = np.zeros((B, H, T, dv))
    S = np.zeros((B, H, dk, dv)) if S0 is None else _np(S0).copy()
    eye = np.eye(dk)
    for b in range(B):
        for t in range(_tokens(lengths, b, T)):
            kt, bt = k[b, :, t], beta[b, :, t, None, None]
            S[b] = np.exp(g[b, :, t, None, None]) * ((eye - bt * kt[:, :, None] * kt[:, None, :]) @ S[b]) \
                + bt * kt[:, :, None] * v[b, :, t, None, :]
            o[b, :, t] = scale * (q[b, :, t, None, :] @ S[b])[:, 0]
    return o, S


def deltarule_backward(q, k, v, g, beta, do, S0=None, dS_T=None, lengths=None, scale=1.0):
    """(dq, dk, dv, dg, dbeta, dS0) by the reverse mode of deltarule_forward, each
    token's from the states before and behind it (all kept)."""
    q, k, v, g, beta, do = _np(q), _np(k), _np(v), _np(g), _np(beta), _np(do)
    B, H, T, dv = v.shape
    Hk, dk = k.shape[1], k.shape[-1]
    q, k = (np.repeat(x, H // Hk, 1) for x in (q, k))
    gq, gk, gv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    gg, gb = np.zeros((B, H, T)), np.zeros((B, H, T))
    D0 = np.zeros((B, H, dk, dv)) if dS_T is None else _np(dS_T).copy()
    eye = np.eye(dk)
    for b in range(B):
        n = _tokens(lengths, b, T)
        S = [np.zeros((H, dk, dv)) if S0 is None else _np(S0)[b]]
        step = []
        for t in range(n):
            kt, bt = k[b, :, t], beta[b, :, t, None, None]
            step.append(eye - bt * kt[:, :, None] * kt[:, None, :])
            S.append(np.exp(g[b, :, t, None, None]) * (step[t] @ S[t]) + bt * kt[:, :, None] * v[b, :, t, None, :])
        D = D0[b]
        for t in range(n - 1, -1, -1):
            kt, bt, vt = k[b, :, t], beta[b, :, t, None], v[b, :, t]
            gam = np.exp(g[b, :, t, None, None])
            gq[b, :, t] = scale * (S[t + 1] @ do[b, :, t, :, None])[..., 0]
            D = D + scale * q[b, :, t, :, None] * do[b, :, t, None, :]
            Dk, Sk = (D.transpose(0, 2, 1) @ kt[..., None])[..., 0], (S[t].transpose(0, 2, 1) @ kt[..., None])[..., 0]
            # L = <D, e^g (S - beta k (k^T S)) + beta k v^T> of this token
            gb[b, :, t] = (Dk * vt).sum(-1) - gam[:, 0, 0] * (Dk * Sk).sum(-1)
            gv[b, :, t] = bt * Dk
            gk[b, :, t] = bt * (D @ vt[..., None])[..., 0] \
                - gam[:, 0] * bt * ((D @ Sk[..., None])[..., 0] + (S[t] @ Dk[..., None])[..., 0])
            gg[b, :, t] = gam[:, 0, 0] * (D * (step[t] @ S[t])).sum((-1, -2))
            D = gam * (step[t] @ D)
        D0[b] = D
    shared = lambda x: x.reshape(B, Hk, H // Hk, T, dk).sum(2)
    return shared(gq), shared(gk), gv, gg, gb, D0


def _qk_turn(x, angle, amp, layout, sign):
    """Rows [B, heads, T, d] with the pairs of their first channels turned by sign * angle [B, T, n]."""
    n = angle.shape[-1]
    y = x.copy()
    c, s = amp * np.cos(angle)[:, None], sign * amp * np.sin(angle)[:, None]
    for i in range(n):
        a, b = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
        y[..., a] = x[..., a] * c[..., i] - x[..., b] * s[..., i]
        y[..., b] = x[..., b] * c[..., i] + x[..., a] * s[..., i]
    return y


def _qk_angle(x, inv_freq, positions):
    B, T = x.shape[0], x.shape[2]
    f = np.zeros(0) if inv_freq is None else _np(inv_freq)
    p = np.broadcast_to(np.arange(T, dtype=np.float64), (B, T)) if positions is None else _np(positions)
    return p[..., None] * f


def _qk_scale(x, norm, eps):
    if norm == "none":
        return np.ones(x.shape[:-1] + (1,))
    sq = (x * x).sum(-1, keepdims=True)
    return 1.0 / np.sqrt((sq / x.shape[-1] if norm == "rms" else sq) + eps)


def qknorm_forward(x, w=None, norm="rms", eps=1e-6, inv_freq=None, positions=None, layout="half", amp=1.0):
    """Norm and rotation of the rows x [B,H,T,d]."""
    x = _np(x)
    z = x * _qk_scale(x, norm, eps) * (1.0 if w is None else _np(w))
    return _qk_turn(z, _qk_angle(x, inv_freq, positions), amp, layout, 1.0)


def qknorm_backward(x, dy, w=None, norm="rms", eps=1e-6, inv_freq=None, positions=None, layout="half", amp=1.0):
    """(dx, dw)."""
    x, dy = _np(x), _np(dy)
    u = _qk_turn(dy, _qk_angle(x, inv_freq, positions), amp, layout, -1.0)
    r = _qk_scale(x, norm, eps)
    dw = (u * x * r).sum((0, 1, 2))
    u = u * (1.0 if w is None else _np(w))
    if norm == "none":
        return u, dw
    n = x.shape[-1] if norm == "rms" else 1
    return r * u - r ** 3 * x * (u * x).sum(-1, keepdims=True) / n, dw


_erf = np.vectorize(math.erf, otypes=[np.float64])


def act(z, name):
    if name == "silu":
        return z / (1.0 + np.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    return z


def act_slope(z, name):
    if name == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return s + z * s * (1.0 - s)
    if name == "gelu":
        return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * np.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
    return np.ones_like(z)


def _axes(over):
    return (3,) if over == "token" else (1, 3)


def groupnorm_forward(x, w=None, b=None, eps=1e-5, name="none", over="token"):
    """(y, mean, rstd) of x [N,S,G,D]; mean, rstd [N,S,G] or [N,G]."""
    x = _np(x)
    w = np.ones(x.shape[2:]) if w is None else _np(w)
    b = np.zeros(x.shape[2:]) if b is None else _np(b)
    m = x.mean(_axes(over), keepdims=True)
    r = 1.0 / np.sqrt(((x - m) ** 2).mean(_axes(over), keepdims=True) + eps)
    y = act((x - m) * r * w + b, name)
    return y, np.squeeze(m, _axes(over)), np.squeeze(r, _axes(over))


def groupnorm_backward(x, dy, mean, rstd, w=None, b=None, name="none", over="token"):
    """(dx, dw, db) with the given statistics taken as those of x."""
    x, dy = _np(x), _np(dy)
    w = np.ones(x.shape[2:]) if w is None else _np(w)
    b = np.zeros(x.shape[2:]) if b is None else _np(b)
    m, r = (np.expand_dims(_np(t), _axes(over)) for t in (mean, rstd))
    xh = (x - m) * r
    dz = dy * act_slope(xh * w + b, name)
    u = dz * w
    dx = r * (u - u.mean(_axes(over), keepdims=True) - xh * (u * xh).mean(_axes(over), keepdims=True))
    return dx, (dz * xh).sum((0, 1)), dz.sum((0, 1))
