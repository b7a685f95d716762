"""The float64 oracles of the gated delta rule and of the norm and rotation of
queries and keys, pinned by differences and by what the formulas say."""
import numpy as np
import pytest

from oracle import ops as O


def data(seed, B=2, Hk=1, H=2, T=7, dk=4, dv=3):
    r = np.random.default_rng(seed)
    n = r.normal
    return dict(q=n(size=(B, Hk, T, dk)), k=n(size=(B, Hk, T, dk)) * 0.5, v=n(size=(B, H, T, dv)),
                g=-np.abs(n(size=(B, H, T))), beta=r.uniform(0, 1, (B, H, T))), n(size=(B, H, dk, dv)), r


def test_delta_rule_with_orthogonal_keys_replaces_what_a_key_holds():
    """beta = 1, no decay, unit keys: writing a key again replaces its value."""
    k = np.zeros((1, 1, 3, 2))
    k[0, 0, 0, 0] = k[0, 0, 1, 1] = k[0, 0, 2, 0] = 1.0
    v = np.arange(1.0, 7.0).reshape(1, 1, 3, 2)
    one = np.ones((1, 1, 3))
    o, S = O.deltarule_forward(k, k, v, 0 * one, one)
    assert np.allclose(S[0, 0], [v[0, 0, 2], v[0, 0, 1]]) and np.allclose(o, v)


def test_delta_rule_without_recall_is_linear_attention():
    """Keys orthogonal to the state and to one another: nothing is taken out."""
    d, S0, r = data(1, H=1, T=4)
    d["k"] = np.broadcast_to(np.eye(4)[None, None], (2, 1, 4, 4)).copy()
    d["g"] = np.full((2, 1, 4), -0.3)
    o, S = O.deltarule_forward(**d)
    want = O.linattn_forward(d["q"], d["k"] * d["beta"][..., None], d["v"], np.array([-0.3]))
    assert np.allclose(o, want[0]) and np.allclose(S, want[1])


@pytest.mark.parametrize("lengths", [None, [7, 3], [0, 9]])
def test_delta_rule_gradients_are_the_differences(lengths):
    d, S0, r = data(2)
    do, dS = r.normal(size=(2, 2, 7, 3)), r.normal(size=S0.shape)
    names = ("q", "k", "v", "g", "beta")

    def loss(x, S):
        o, ST = O.deltarule_forward(*(x[n] for n in names), S, lengths, 0.7)
        return (o * do).sum() + (ST * dS).sum()

    got = O.deltarule_backward(*(d[n] for n in names), do, S0, dS, lengths, 0.7)
    e = 1e-6
    for name, gr in zip(names + ("S0",), got):
        t = S0 if name == "S0" else d[name]
        num = np.zeros_like(t)
        for i in np.ndindex(t.shape):
            old = t[i]
            t[i] = old + e
            up = loss(d, S0)
            t[i] = old - e
            num[i] = (up - loss(d, S0)) / (2 * e)
            t[i] = old
        # second differences of a loss of order 10: e^2 and 2^-52 * 10 / e
        assert np.max(np.abs(num - gr)) < 1e-7, name


@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_rotation_keeps_lengths_and_depends_on_distance(layout):
    r = np.random.default_rng(3)
    q, k = r.normal(size=(1, 1, 1, 6)), r.normal(size=(1, 1, 1, 6))
    f = np.array([1.0, 0.1])
    at = lambda x, p: O.qknorm_forward(x, norm="none", inv_freq=f, positions=np.array([[p]]), layout=layout)
    assert np.allclose((at(q, 12345) ** 2).sum(), (q ** 2).sum())
    assert np.allclose(at(q, 0), q)
    assert np.isclose((at(q, 1007) * at(k, 1000)).sum(), (at(q, 7) * at(k, 0)).sum())
    one = O.qknorm_forward(np.eye(6)[0].reshape(1, 1, 1, 6), norm="none", inv_freq=f, positions=np.array([[0.5]]),
                           layout=layout)[0, 0, 0]
    b = 2 if layout == "half" else 1
    assert np.isclose(one[0], np.cos(0.5)) and np.isclose(one[b], np.sin(0.5))


@pytest.mark.parametrize("norm", ["none", "rms", "l2"])
def test_norm_and_its_gradients(norm):
    r = np.random.default_rng(4)
    x, w, dy = r.normal(size=(2, 2, 3, 5)), r.normal(size=5), r.normal(size=(2, 2, 3, 5))
    kw = dict(norm=norm, eps=1e-3, inv_freq=np.array([0.7, 0.2]), layout="half", amp=1.3)
    if norm != "none":
        y = O.qknorm_forward(x, None, norm, 0.0)
        assert np.allclose((y * y).sum(-1), 5.0 if norm == "rms" else 1.0)
    loss = lambda: (O.qknorm_forward(x, w, **kw) * dy).sum()
    dx, dw = O.qknorm_backward(x, dy, w, **kw)
    for t, gr in ((x, dx), (w, dw)):
        for i in np.ndindex(t.shape):
            old = t[i]
            t[i] = old + 1e-6
            up = loss()
            t[i] = old - 1e-6
            num = (up - loss()) / 2e-6
            t[i] = old
            assert abs(num - gr[i]) < 1e-7
