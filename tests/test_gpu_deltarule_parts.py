"""What bfloat16 calls of the gated delta rule keep of values that are split into bfloat16
parts, on inputs where a part less shows.

States that are handed out and the gates' gradients: three parts, float32 sums.  Keys are unit
vectors (one +-1 each) and decays 1, so that every product with a key is exact and few terms meet.
U = 2^-24; A is a result's own sum of magnitudes.  On the way to a state's element:
v - S^T k one rounding; an inverse's entry times beta one; its three parts times the right
side's three without the products past the third order (2 parts of 2^-7 2^-15: 8 U) and six
accumulations in the matrix unit (2 U each); three accumulations into S (2 U each): 28 U, taken as
40.  Of a value in two parts up to 2^-16 is lost, 256 U.
dbeta is a product of two such results, 2 * 40 + 16 U.  dlog_decay of a single token is a sum of
five products of them, one of which goes through the matrix unit in three parts: 32 U.

Results in bfloat16: 2^-8 of themselves, and of A 2^-16 for each operand in two parts,
2^-14 where two such meet (the product of their second parts is left out) and 2^-15 where the second of
three cut parts is the last one used, besides (4 d_qk + 64) U for float32 sums.
"""
import numpy as np
import pytest
import torch

from oracle import ops as O
from xlstm_mlstm_matrix_amd import binding as B

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
NAMES = ("q", "k", "v", "g", "beta")


def magnitudes(d, scale):
    """The recurrences on the magnitudes of all inputs with every sign positive."""
    f = {n: np.abs(O._np(x)) for n, x in d.items() if n != "g"}
    gam = np.exp(O._np(d["g"]))
    q, k, v, beta, do = (f[n] for n in ("q", "k", "v", "beta", "do"))
    T = v.shape[2]
    left = lambda a, M: (a[:, :, None, :] @ M)[:, :, 0]
    right = lambda M, a: (M @ a[..., None])[..., 0]
    outer = lambda a, c: a[..., None] * c[:, :, None, :]
    S, before, x, o = f["S0"], [], [], []
    for t in range(T):
        S = gam[:, :, t, None, None] * S
        before.append(S)
        x.append(v[:, :, t] + left(k[:, :, t], S))
        S = S + outer(k[:, :, t], beta[:, :, t, None] * x[t])
        o.append(scale * left(q[:, :, t], S))
    w = {"S": S, "o": np.stack(o, 2)}
    D, rows = f["dS"], {n: [None] * T for n in ("dq", "dk", "dv", "dbeta", "dlog", "tail")}
    for t in range(T - 1, -1, -1):
        bt = beta[:, :, t, None]
        after = before[t] + outer(k[:, :, t], bt * x[t])
        rows["dq"][t] = scale * right(after, do[:, :, t])
        # dlog_decay as (do.o + dv.v)_t + <D, S> with S written as what the token found and added
        rows["dlog"][t] = (rows["dq"][t] * q[:, :, t]).sum(-1) + (D * after).sum((-1, -2))
        D = D + scale * outer(q[:, :, t], do[:, :, t])
        du = left(k[:, :, t], D)
        rows["dv"][t] = bt * du
        rows["dlog"][t] += (rows["dv"][t] * v[:, :, t]).sum(-1)
        rows["dk"][t] = right(D, bt * x[t]) + right(before[t], bt * du)
        rows["dbeta"][t] = (du * x[t]).sum(-1)
        D = gam[:, :, t, None, None] * (D + outer(k[:, :, t], bt * du))
    w.update({n: np.stack(rows[n], 2) for n in ("dq", "dk", "dv", "dbeta", "dlog")}, dS0=D)
    return w


def unit_keys(r, cells, T, dk, spread):
    """One +-1 in each row: `spread` channels first, then some of them again."""
    k = np.zeros((*cells, T, dk), np.float32)
    for i in np.ndindex(cells):
        for c in range(0, T, 24):     # anew for every 24 tokens
            n = min(24, T - c)
            ch = r.permutation(dk)[:min(n, spread)]
            ch = np.concatenate([ch, r.permutation(ch)[:n - len(ch)]])
            k[(*i, np.arange(c, c + n), ch)] = r.choice([-1.0, 1.0], n)
    return k


def case(seed, cells, T, dk, dv, spread=16, columns=None):
    r = np.random.default_rng(seed)
    n = lambda *s: r.normal(0, 1, s).astype(np.float32)
    keep = np.zeros(dv, np.float32)
    keep[slice(None) if columns is None else columns] = 1.0
    d = {"q": np.zeros((*cells, T, dk), np.float32), "k": unit_keys(r, cells, T, dk, spread), "v": 0.25 * n(*cells, T, dv) * keep,
         "g": np.zeros((*cells, T), np.float32), "beta": r.uniform(0.02, 1.0, (*cells, T)).astype(np.float32),
         "do": np.zeros((*cells, T, dv), np.float32), "S0": n(*cells, dk, dv) * keep, "dS": n(*cells, dk, dv) * keep}
    d = {x: torch.from_numpy(t) for x, t in d.items()}
    return {x: t.bfloat16() if x in ("q", "k", "v", "do") else t for x, t in d.items()}


def both(d, scale=1.0, state=True):
    g = {n: x.cuda() for n, x in d.items()}
    a = [g[n] for n in NAMES]
    o = B.deltarule_fwd(*a, g["S0"], scale=scale, return_state=state)
    back = B.deltarule_bwd(*a, g["do"], g["S0"], g["dS"], scale=scale, state_grad=True)
    torch.cuda.synchronize()
    got = dict(zip(("dq", "dk", "dv", "dlog", "dbeta", "dS0"), back))
    got["o"], got["S"] = o if state else (o, None)
    c = [O._np(d[n]) for n in NAMES]
    ro, rS = O.deltarule_forward(*c, d["S0"], None, scale)
    ref = dict(zip(("dq", "dk", "dv", "dlog", "dbeta", "dS0"), O.deltarule_backward(*c, d["do"], d["S0"], d["dS"], None, scale)))
    ref.update(o=ro, S=rS)
    return got, ref, magnitudes(d, scale)


def close(x, ref, tol, what):
    err = np.abs(x.detach().double().cpu().numpy() - ref)
    bad = float((err / (tol + 1e-30)).max())
    print(f"[delta] {what}: {bad:.3f} of the bound", flush=True)
    assert bad <= 1.0, (what, bad)


@pytest.mark.parametrize("T", [1, 24, 72])
@pytest.mark.parametrize("dk,dv", [(32, 64), (128, 128), (256, 80)])
def test_states_are_float32_sums(T, dk, dv):
    got, ref, A = both(case(T + dk, (2, 3), T, dk, dv))
    for n in ("S", "dS0"):
        close(got[n], ref[n], 40 * U * -(-T // 24) * A[n], f"{n} of {T} tokens, {dk} x {dv}")


def test_states_are_float32_sums_with_128_columns():
    """The same in a call of 256 heads."""
    got, ref, A = both(case(5, (16, 16), 24, 64, 64))
    for n in ("S", "dS0"):
        close(got[n], ref[n], 40 * U * A[n], f"{n} of 256 heads")


@pytest.mark.parametrize("T", [1, 24])
@pytest.mark.parametrize("dk", [32, 256])
def test_dbeta_is_a_float32_sum(T, dk):
    """A single column of values: what dU and X lose does not average out."""
    got, ref, A = both(case(T + dk, (4, 8), T, dk, 16, columns=5))
    close(got["dbeta"], ref["dbeta"], 96 * U * A["dbeta"], f"dbeta of {T} tokens, {dk}")


@pytest.mark.parametrize("heads", [(4, 16), (16, 16)], ids=["64", "128 columns"])
def test_dlog_decay_is_a_float32_sum(heads):
    """Single tokens whose query, key and states share one element, of magnitudes that let each
    term of the sum be the largest in some of them."""
    d = case(3, heads, 1, 16, 16, columns=5)
    r = np.random.default_rng(4)
    size = lambda: torch.from_numpy(np.exp2(r.uniform(-6, 2, heads)).astype(np.float32))
    d["q"] = d["k"].clone()
    hit = d["k"][:, :, 0].float().abs()[..., None]
    d["S0"], d["dS"] = d["S0"] * hit * size()[..., None, None], d["dS"] * hit * size()[..., None, None]
    d["v"] = (d["v"].float() * size()[..., None, None]).bfloat16()
    d["do"][..., 5] = (size() * torch.from_numpy(r.choice([-1.0, 1.0], heads).astype(np.float32)))[..., None].bfloat16()
    d["beta"] = torch.from_numpy(np.exp2(r.uniform(-6, 0, (*heads, 1))).astype(np.float32))
    got, ref, A = both(d, scale=0.7)
    close(got["dlog"], ref["dlog"], 32 * U * A["dlog"], f"dlog_decay of {heads}")


@pytest.mark.parametrize("shape", [(2, 3, 1, 16, 32), (2, 3, 2, 16, 64), (1, 4, 6, 32, 64), (1, 2, 7, 128, 128),
                                   (1, 2, 5, 240, 64), (16, 16, 3, 16, 64)], ids=str)
@pytest.mark.parametrize("state", [True, False])
def test_bfloat16_outputs_are_rounded_once(shape, state):
    """Where a sum's terms cancel an operand with a part less is far past this bound."""
    cells, T, dk, dv = shape[:2], *shape[2:]
    r = np.random.default_rng(sum(shape))
    n = lambda *s: torch.from_numpy(r.normal(0, 1, s).astype(np.float32))
    unit = lambda *s: torch.nn.functional.normalize(n(*s), dim=-1)
    d = {"q": unit(*cells, T, dk).bfloat16(), "k": unit(*cells, T, dk).bfloat16(), "v": n(*cells, T, dv).bfloat16(),
         "do": n(*cells, T, dv).bfloat16(), "g": -0.1 * n(*cells, T).abs(), "beta": torch.sigmoid(n(*cells, T)),
         "S0": n(*cells, dk, dv), "dS": n(*cells, dk, dv)}
    got, ref, A = both(d, scale=dk ** -0.5, state=state)
    own = 1.01 * 2.0 ** -8
    f32 = (4 * dk + 64) * U
    # o: S, P and U (without a state handed out also S's own copy for the keys, the inverse and the right side)
    part = {"o": (3 if state else 6) * 2.0 ** -16 + 2.0 ** -14 * (1 if state else 3), "dq": 2 * 2.0 ** -16, "dv": 0.0,
            "dk": 4 * 2.0 ** -16 + 2 * (2.0 ** -14 + 2.0 ** -15)}
    for name, p in part.items():
        close(got[name], ref[name], own * np.abs(ref[name]) + (p + f32) * A[name], f"{shape} state {state} {name}")
