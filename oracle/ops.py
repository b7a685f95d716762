"""float64 oracle of linear attention with a decay for each head and of group
norm with an activation, written token by token and row by row from the
formulas (numpy; shares nothing with the HIP kernels).

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
