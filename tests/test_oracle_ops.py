"""The float64 oracle of linear attention and group norm: its gradients
against differences of its forward, and the recurrence against the unrolled sum."""
import numpy as np
import pytest

from oracle import ops as O


def rnd(seed, *shape):
    return np.random.default_rng(seed).normal(size=shape)


def numgrad(f, x, h=1e-5):
    """Central differences of a scalar function; their error is O(h^2) + O(1e-16 / h)."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        s = x[i]
        x[i] = s + h
        a = f()
        x[i] = s - h
        b = f()
        x[i] = s
        g[i] = (a - b) / (2 * h)
    return g


def test_linattn_unrolled():
    q, k, v, S0 = rnd(0, 2, 2, 7, 3), rnd(1, 2, 2, 7, 3), rnd(2, 2, 2, 7, 4), rnd(3, 2, 2, 3, 4)
    g = np.array([-0.3, -np.inf])
    o, S = O.linattn_forward(q, k, v, g, S0, scale=0.5)
    gam = np.exp(g)
    for h in range(2):
        for t in range(7):
            r = gam[h] ** (t + 1) * S0[:, h]
            for j in range(t + 1):
                r = r + gam[h] ** (t - j) * k[:, h, j, :, None] * v[:, h, j, None, :]
            np.testing.assert_allclose(o[:, h, t], 0.5 * np.einsum("bk,bkv->bv", q[:, h, t], r), atol=1e-12)
        np.testing.assert_allclose(S[:, h], r, atol=1e-12)


@pytest.mark.parametrize("lengths", [None, [4, 0]])
def test_linattn_gradients(lengths):
    x = {n: rnd(i, 2, 2, 5, 3) for i, n in enumerate("qk")}
    x["v"], x["S0"] = rnd(5, 2, 2, 5, 2), rnd(6, 2, 2, 3, 2)
    do, dS = rnd(7, 2, 2, 5, 2), rnd(8, 2, 2, 3, 2)
    g = np.array([-0.2, -1.5])

    def loss():
        o, S = O.linattn_forward(x["q"], x["k"], x["v"], g, x["S0"], lengths, 0.7)
        return (o * do).sum() + (S * dS).sum()

    got = O.linattn_backward(x["q"], x["k"], x["v"], g, do, x["S0"], dS, lengths, 0.7)
    for n, r in zip(("q", "k", "v", "S0"), got):
        np.testing.assert_allclose(numgrad(loss, x[n]), r, atol=1e-7, err_msg=n)


@pytest.mark.parametrize("over", ["token", "sequence"])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_groupnorm_gradients(over, act):
    x, w, b, dy = rnd(0, 2, 3, 2, 4), rnd(1, 2, 4), rnd(2, 2, 4), rnd(3, 2, 3, 2, 4)

    def loss():
        return (O.groupnorm_forward(x, w, b, 1e-2, act, over)[0] * dy).sum()

    _, m, r = O.groupnorm_forward(x, w, b, 1e-2, act, over)
    dx, dw, db = O.groupnorm_backward(x, dy, m, r, w, b, act, over)
    for n, p, ref in (("x", x, dx), ("w", w, dw), ("b", b, db)):
        np.testing.assert_allclose(numgrad(loss, p), ref, atol=1e-7, err_msg=n)


def test_groupnorm_moments():
    x = rnd(4, 2, 6, 3, 5) + 2.0
    for over, ax in (("token", 3), ("sequence", (1, 3))):
        y, m, r = O.groupnorm_forward(x, over=over, eps=1e-9)
        np.testing.assert_allclose(y.mean(ax), 0.0, atol=1e-12)
        np.testing.assert_allclose(y.var(ax), 1.0, atol=1e-8)
        np.testing.assert_allclose(m, x.mean(ax), atol=1e-12)
