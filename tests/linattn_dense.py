"""Linear attention in its unrolled form, float64 on the CPU: every output as one
masked product over all earlier tokens, gradients by differentiating that.  Much
faster than the recurrence token by token, so it serves many and large shapes;
test_linattn_dense.py holds the two to each other."""
import torch


def _power(g, steps):
    """e^{g steps}, 1 for no steps (g may be -inf)."""
    return torch.where(steps == 0, torch.ones_like(steps), torch.exp(g[:, None] * steps.reshape(1, -1).clamp(min=1)).reshape(
        len(g), *steps.shape))


def forward(q, k, v, g, S0=None, lengths=None, scale=1.0):
    """(o, S_T), differentiable in q, k, v and S0."""
    B, H, T, _ = q.shape
    os, Ss = [], []
    for b in range(B):
        n = T if lengths is None else min(max(int(lengths[b]), 0), T)
        t = torch.arange(n, dtype=torch.float64)
        dist = t[:, None] - t[None, :]
        dec = _power(g, dist.clamp(min=0)) * (dist >= 0)
        o = (q[b, :, :n] @ k[b, :, :n].transpose(-1, -2) * dec) @ v[b, :, :n]
        S = (k[b, :, :n] * _power(g, n - 1 - t)[..., None]).transpose(-1, -2) @ v[b, :, :n]
        if S0 is not None:
            o = o + (q[b, :, :n] @ S0[b]) * _power(g, t + 1)[..., None]
            S = S + S0[b] * _power(g, torch.tensor([float(n)], dtype=torch.float64))[..., None]
        os.append(torch.cat([scale * o, torch.zeros((H, T - n, v.shape[-1]), dtype=torch.float64)], 1))
        Ss.append(S)
    return torch.stack(os), torch.stack(Ss)


def both(d, lengths=None, scale=1.0, magnitudes=False):
    """(o, S_T), (dq, dk, dv, dS0) of the inputs d (q, k, v, g, S0, do, dS), or of
    their magnitudes."""
    x = {n: None if t is None else t.double() for n, t in d.items()}
    if magnitudes:
        x = {n: t if t is None or n == "g" else t.abs() for n, t in x.items()}
    if x["S0"] is None:
        x["S0"] = torch.zeros(x["q"].shape[:2] + (x["q"].shape[3], x["v"].shape[3]), dtype=torch.float64)
    leaf = [x[n].requires_grad_() for n in ("q", "k", "v", "S0")]
    out = forward(*leaf[:3], x["g"], leaf[3], lengths, abs(scale) if magnitudes else scale)
    loss = (out[0] * x["do"]).sum()
    if x["dS"] is not None:
        loss = loss + (out[1] * x["dS"]).sum()
    return [t.detach().numpy() for t in out], [t.numpy() for t in torch.autograd.grad(loss, leaf)]
