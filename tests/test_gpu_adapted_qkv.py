"""AdaptedQKV: projection with adapters, then rotary positions, as a model runs them,
against the same chain in float64 on the CPU.

Bounds (derived before any run): the packed projection is a bf16 value (2^-8 of itself
allowed, with the low-rank and accumulation parts of its own bound), a rotation mixes
two of them (|x1| + |x2| of those errors) and rounds once more (2^-8)."""
import numpy as np
import pytest
import torch

from gpu_util import dev, status_of, status_tensor
from test_gpu_lora import bf, get, put

pytestmark = pytest.mark.gpu

HID, NQ, NKV, D, L, R = 256, 4, 2, 32, 3, 16


@pytest.fixture(scope="module")
def gg():
    import __graft_entry__ as g
    g.build()
    import unpermute_route_hist_gb300 as gg
    return gg


def weights(seed=0):
    g = np.random.default_rng(seed)
    N = (NQ + 2 * NKV) * D
    return dict(W=bf(g.standard_normal((N, HID)) * 0.06), A=bf(g.standard_normal((L, R, HID)) * 0.06),
                B=bf(g.standard_normal((L, N, R)) * 0.1), scale=g.uniform(0.5, 2.0, L).astype(np.float32))


def turn(x, pos, inv, sign):
    """Rotary positions on the q and k heads of packed rows [T, heads, D], halves paired."""
    h = len(inv)
    th = pos[:, None].astype(np.float64) * inv
    c, s = np.cos(th)[:, None], sign * np.sin(th)[:, None]
    y = x.copy()
    qk = slice(0, NQ + NKV)
    a, b = x[:, qk, :h], x[:, qk, h:2 * h]
    y[:, qk, :h], y[:, qk, h:2 * h] = a * c - b * s, b * c + a * s
    return y


def pairwise(e, h):
    """Of each element of a turned pair, the sum of both elements' values."""
    y = e.copy()
    qk = slice(0, NQ + NKV)
    y[:, qk, :h] = y[:, qk, h:2 * h] = e[:, qk, :h] + e[:, qk, h:2 * h]
    return y


def layer(gg, w, rot):
    from unpermute_route_hist_gb300.adapters import AdaptedQKV
    freqs = gg.rope_freqs(rot, device=dev())
    return AdaptedQKV(put(w["W"]), put(w["A"]), put(w["B"]), torch.from_numpy(w["scale"]).to(dev()), NQ, NKV, D, freqs)


@pytest.mark.parametrize("T,rot", [(1, 32), (37, 16), (300, 32)])
def test_forward_and_backward(gg, T, rot):
    from unpermute_route_hist_gb300 import rotary
    w = weights()
    g = np.random.default_rng(T)
    X, dY = bf(g.standard_normal((T, HID))), bf(g.standard_normal((T, w["W"].shape[0])))
    ids, pos = g.integers(-1, L, T).astype(np.int32), g.integers(0, 5000, T).astype(np.int32)
    inv = rotary.frequencies(rot)[0]
    m, st = layer(gg, w, rot), status_tensor()
    plan = gg.lora_plan(torch.from_numpy(ids).to(dev()), L, status=st)
    q, k, v, saved = m.forward(put(X), plan, torch.from_numpy(pos).to(dev()), status=st)
    # forward
    U = np.zeros((T, R))
    base, err = X @ w["W"].T, 2.0 ** -14 * (np.abs(X) @ np.abs(w["W"]).T)
    for a in range(L):
        i = np.flatnonzero(ids == a)
        U[i] = w["scale"][a] * (X[i] @ w["A"][a].T)
        mag = w["scale"][a] * (np.abs(X[i]) @ np.abs(w["A"][a]).T)
        base[i] += U[i] @ w["B"][a].T
        err[i] += (2.0 ** -8 * np.abs(U[i]) + 2.0 ** -13 * mag) @ np.abs(w["B"][a]).T
    err += 2.0 ** -8 * np.abs(base)
    heads = lambda z: z.reshape(T, NQ + 2 * NKV, D)
    want = turn(heads(base), pos, inv, 1.0)
    bound = pairwise(heads(err), rot // 2) + 2.0 ** -8 * pairwise(np.abs(heads(base)), rot // 2)
    got = np.concatenate([get(q), get(k), get(v)], axis=1)
    assert (np.abs(got - want) <= bound).all()
    # backward: the gradient enters turned back and rounded to bf16
    dX, dA, dB = m.backward(put(dY), saved, status=st)
    assert status_of(st) == 0
    back = turn(heads(dY), pos, inv, -1.0).reshape(T, -1)
    eback = 2.0 ** -8 * pairwise(np.abs(heads(dY)), rot // 2).reshape(T, -1)
    wX, eX = back @ w["W"], (eback + 2.0 ** -14 * np.abs(back)) @ np.abs(w["W"])
    for a in range(L):
        i = np.flatnonzero(ids == a)
        V = w["scale"][a] * (back[i] @ w["B"][a])
        eV = w["scale"][a] * ((eback[i] + 2.0 ** -14 * np.abs(back[i])) @ np.abs(w["B"][a]))
        wX[i] += V @ w["A"][a]
        eX[i] += (eV + (2.0 ** -8 + 2.0 ** -14) * np.abs(V)) @ np.abs(w["A"][a])
        rA, rB = V.T @ X[i], back[i].T @ U[i]
        eA = (eV + 2.0 ** -13 * np.abs(V)).T @ np.abs(X[i]) + 2.0 ** -8 * np.abs(rA)
        eU = 2.0 ** -8 * np.abs(U[i]) + 2.0 ** -13 * w["scale"][a] * (np.abs(X[i]) @ np.abs(w["A"][a]).T)
        eB = (eback[i] + 2.0 ** -13 * np.abs(back[i])).T @ (np.abs(U[i]) + eU) + np.abs(back[i]).T @ eU + 2.0 ** -8 * np.abs(rB)
        assert (np.abs(get(dA)[a] - rA) <= eA + 1e-30).all() and (np.abs(get(dB)[a] - rB) <= eB + 1e-30).all()
    assert (np.abs(get(dX) - wX) <= eX + 2.0 ** -8 * np.abs(wX) + 1e-30).all()


def test_decoding_continues_a_prefill(gg):
    """A prompt in one call and the same tokens one by one give the same heads, to the
    bf16 rounding of sums taken in another order (2^-7 of the value, 2^-12 of the
    projection's magnitude)."""
    w = weights(1)
    m = layer(gg, w, 32)
    g = np.random.default_rng(2)
    X = bf(g.standard_normal((9, HID)))
    ids = np.full(9, 1, np.int32)
    pos = np.arange(100, 109, dtype=np.int32)
    one = lambda s: m.forward(put(X[s]), gg.lora_plan(torch.from_numpy(ids[s]).to(dev()), L), torch.from_numpy(pos[s]).to(dev()))
    whole = [get(t) for t in one(slice(0, 9))[:3]]
    mag = float(np.abs(whole[0]).max() + np.abs(whole[1]).max())
    for t in range(9):
        step = [get(x) for x in one(slice(t, t + 1))[:3]]
        for a, b in zip(whole, step):
            assert (np.abs(a[t] - b[0]) <= 2.0 ** -6 * np.abs(b[0]) + 2.0 ** -7 * mag * 2.0 ** -1).all()


def test_refuses_what_does_not_fit(gg):
    from unpermute_route_hist_gb300.adapters import AdaptedQKV
    w = weights()
    with pytest.raises(ValueError):
        AdaptedQKV(put(w["W"][:-D]), put(w["A"]), put(w["B"]), None, NQ, NKV, D, None)
    with pytest.raises(ValueError):
        AdaptedQKV(put(w["W"]), put(w["A"]), put(w["B"]), None, NQ, NKV, D, gg.rope_freqs(2 * D, device=dev()))
