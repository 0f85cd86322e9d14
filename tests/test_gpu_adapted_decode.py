"""AdaptedQKV: a prompt in one call and its tokens one by one, each against the chain in float64 and
each against the other, element by element.

Bounds (derived before any run).  The packed projection of a call is a bf16 value: 2^-8 of itself
allowed, U's rounding (2^-8 of |U|) and U's sums (2^-14 of the terms' magnitudes) through |B|, and
2^-14 of the shared terms' magnitudes (at most 1024 terms).  A rotation mixes two elements: the sum of
both elements' errors, then one more rounding (2^-8).  Two calls differ by at most twice that."""
import numpy as np
import pytest
import torch

from gpu_util import dev, status_of, status_tensor
from test_gpu_adapted_qkv import D, HID, L, NKV, NQ, layer, pairwise, turn, weights
from test_gpu_lora import bf, get, put

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gg():
    import __graft_entry__ as g
    g.build()
    import unpermute_route_hist_gb300 as gg
    return gg


@pytest.mark.parametrize("T,rot,adapter", [(9, 32, 1), (70, 16, 0), (9, 32, -1)])
def test_decoding_gives_the_prefills_heads(gg, T, rot, adapter):
    from unpermute_route_hist_gb300 import rotary
    w, st = weights(1), status_tensor()
    m = layer(gg, w, rot)
    X = bf(np.random.default_rng(2).standard_normal((T, HID)))
    ids, pos = np.full(T, adapter, np.int32), np.arange(100, 100 + T, dtype=np.int32)
    inv = rotary.frequencies(rot)[0]
    put_int = lambda x: torch.from_numpy(x).to(dev())

    def heads(s):
        out = m.forward(put(X[s]), gg.lora_plan(put_int(ids[s]), L, status=st), put_int(pos[s]), status=st)
        return np.concatenate([get(t) for t in out[:3]], axis=1)

    base, err = X @ w["W"].T, 2.0 ** -14 * (np.abs(X) @ np.abs(w["W"]).T)
    if adapter >= 0:
        U = w["scale"][adapter] * (X @ w["A"][adapter].T)
        mag = w["scale"][adapter] * (np.abs(X) @ np.abs(w["A"][adapter]).T)
        base = base + U @ w["B"][adapter].T
        err += (2.0 ** -8 * np.abs(U) + 2.0 ** -14 * mag + 2.0 ** -14 * np.abs(U)) @ np.abs(w["B"][adapter]).T
    err += 2.0 ** -8 * np.abs(base)
    split = lambda z: z.reshape(T, NQ + 2 * NKV, D)
    want = turn(split(base), pos, inv, 1.0)
    # the turned elements: the pair's errors, a rounding, and 2^-21 of the pair for cos and sin; the others: their own
    bound = pairwise(split(err), rot // 2) + 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * pairwise(np.abs(split(base)), rot // 2)
    whole = heads(slice(0, T))
    ones = np.concatenate([heads(slice(t, t + 1)) for t in range(T)])
    assert status_of(st) == 0
    for got in (whole, ones):
        assert (np.abs(got - want) <= bound).all(), float((np.abs(got - want) / bound).max())
    assert (np.abs(whole - ones) <= 2 * bound).all()
