"""Host side of the adapter and rotary entry points: sizes, refusals and empty problems.
No call here reaches the GPU (each returns before any CUDA work); and the frequency
table against its definition."""
import ctypes
import math

import numpy as np
import pytest


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    from unpermute_route_hist_gb300 import _lib
    return _lib.load()


fake = ctypes.c_void_p(4096)  # never dereferenced: every call below fails validation first
odd = ctypes.c_void_p(4096 + 2)


def test_plan_size(lib):
    size = lib.gg_lora_plan_size
    assert size(0, 8) > 0 and size(-1, 8) == 0 and size(8, 0) == 0 and size(8, 2049) == 0
    # a mask of 256 bits for each of min(L, 256) adapters of each 256 rows, and the rows' order
    assert size(8192, 64) >= 32 * 64 * 32 + 8192 * 4
    assert size(8192, 64) % 256 == 0 and size(8192, 64) < size(8192, 65) < size(8448, 65)


def test_plan_refusals(lib):
    from unpermute_route_hist_gb300 import _lib
    need = lib.gg_lora_plan_size(100, 4)
    assert lib.gg_lora_plan(fake, -1, 4, fake, need, None, None) == _lib.GG_ERR_INVALID_ARG
    assert lib.gg_lora_plan(fake, 100, 0, fake, need, None, None) == _lib.GG_ERR_INVALID_ARG
    assert lib.gg_lora_plan(fake, 100, 2049, fake, need, None, None) == _lib.GG_ERR_UNSUPPORTED
    assert lib.gg_lora_plan(None, 100, 4, fake, need, None, None) == _lib.GG_ERR_INVALID_ARG
    assert lib.gg_lora_plan(fake, 100, 4, fake, need - 1, None, None) == _lib.GG_ERR_WORKSPACE
    assert lib.gg_lora_plan(fake, 100, 4, odd, need, None, None) == _lib.GG_ERR_WORKSPACE
    assert lib.gg_lora_plan(None, 0, 4, None, 0, None, None) == _lib.GG_OK


def forward(lib, X=fake, W=fake, A=fake, B=fake, plan=fake, T=4, L=2, r=8, N=16, K=24, Y=fake, U=fake):
    return lib.gg_lora_forward(X, W, A, B, None, plan, T, L, r, N, K, Y, U, None, None)


def test_forward_refusals(lib):
    from unpermute_route_hist_gb300 import _lib
    for bad in (dict(T=-1), dict(L=0), dict(r=0), dict(N=-8), dict(K=-8), dict(X=None), dict(W=None), dict(A=None),
                dict(B=None), dict(plan=None), dict(Y=None), dict(U=None)):
        assert forward(lib, **bad) == _lib.GG_ERR_INVALID_ARG, bad
    for bad in (dict(r=12), dict(r=264), dict(N=20), dict(K=28), dict(L=2049), dict(T=2 ** 31 - 1), dict(X=odd),
                dict(W=odd), dict(A=odd), dict(B=odd), dict(Y=odd), dict(U=odd), dict(plan=odd)):
        assert forward(lib, **bad) == _lib.GG_ERR_UNSUPPORTED, bad
    assert forward(lib, T=0, X=None, Y=None, U=None, plan=None) == _lib.GG_OK


def backward(lib, dY=fake, X=fake, W=fake, A=fake, B=fake, plan=fake, U=fake, T=4, L=2, r=8, N=16, K=24, dX=fake,
             dA=fake, dB=fake, ws=fake, nbytes=None):
    nbytes = lib.gg_lora_backward_workspace_size(T, r) if nbytes is None else nbytes
    return lib.gg_lora_backward(dY, X, W, A, B, None, plan, U, T, L, r, N, K, dX, dA, dB, ws, nbytes, None, None)


def test_backward_refusals(lib):
    from unpermute_route_hist_gb300 import _lib
    need = lib.gg_lora_backward_workspace_size(4, 8)
    assert need > 2 * 4 * 8 * 2 and lib.gg_lora_backward_workspace_size(-1, 8) == 0
    for bad in (dict(T=-1), dict(r=-8), dict(dY=None), dict(B=None), dict(W=None), dict(A=None), dict(X=None),
                dict(U=None), dict(plan=None), dict(X=None, dX=None, dB=None), dict(U=None, dX=None, dA=None)):
        assert backward(lib, nbytes=need, **bad) == _lib.GG_ERR_INVALID_ARG, bad
    for bad in (dict(r=20), dict(N=12), dict(dX=odd), dict(dA=odd), dict(dB=odd), dict(dY=odd), dict(X=odd)):
        assert backward(lib, nbytes=10 ** 9, **bad) == _lib.GG_ERR_UNSUPPORTED, bad
    for bad in (dict(ws=None), dict(ws=odd), dict(nbytes=need - 1)):
        assert backward(lib, **bad) == _lib.GG_ERR_WORKSPACE, bad
    assert backward(lib, dX=None, dA=None, dB=None, dY=None) == _lib.GG_OK  # nothing wanted


def rope(lib, q=fake, n_q=2, k=None, n_k=0, out_q=fake, out_k=None, pos=fake, axes=1, sec=None, steps=fake, T=3, D=16,
         rot=8, dtype=0, qt=32, qh=16, ot=32, oh=16):
    arr = (ctypes.c_int32 * len(sec))(*sec) if sec else None
    return lib.gg_rope(q, qt, qh, n_q, k, 32, 16, n_k, out_q, ot, oh, out_k, 32, 16, pos, axes, arr, steps, 1.0, T, D, rot,
                       0, dtype, 0, None)


def test_rope_refusals(lib):
    from unpermute_route_hist_gb300 import _lib
    for bad in (dict(T=-1), dict(D=-1), dict(rot=-2), dict(rot=7), dict(rot=18), dict(n_q=-1), dict(axes=0), dict(axes=5),
                dict(axes=2), dict(axes=2, sec=(1, 2)), dict(axes=2, sec=(-1, 5)), dict(dtype=3), dict(q=None),
                dict(out_q=None), dict(pos=None), dict(steps=None), dict(n_k=1), dict(qt=-1)):
        assert rope(lib, **bad) == _lib.GG_ERR_INVALID_ARG, bad
    assert rope(lib, rot=2048, D=2048) == _lib.GG_ERR_UNSUPPORTED
    assert rope(lib, n_q=70000) == _lib.GG_ERR_UNSUPPORTED
    assert rope(lib, q=ctypes.c_void_p(4097)) == _lib.GG_ERR_UNSUPPORTED      # not on an element
    assert rope(lib, q=odd, out_q=odd, dtype=2) == _lib.GG_ERR_UNSUPPORTED
    assert rope(lib, T=0, q=None) == _lib.GG_OK and rope(lib, n_q=0, q=None) == _lib.GG_OK
    assert rope(lib, rot=0) == _lib.GG_OK                                     # in place with nothing to turn


def test_frequencies():
    from unpermute_route_hist_gb300 import rotary
    inv, m = rotary.frequencies(8, 100.0)
    np.testing.assert_allclose(inv, [1.0, 100 ** -0.25, 0.1, 100 ** -0.75], rtol=1e-15)
    assert m == 1.0
    np.testing.assert_allclose(rotary.frequencies(8, 100.0, "linear", 4.0)[0], inv / 4, rtol=1e-15)
    # ntk: the fastest pair as it was, the slowest stretched by the factor
    ntk = rotary.frequencies(8, 100.0, "ntk", 4.0)[0]
    assert ntk[0] == 1.0 and math.isclose(ntk[-1], inv[-1] / 4, rel_tol=1e-12)
    # yarn: many turns over the trained length keep their speed, less than one is interpolated
    y, m = rotary.frequencies(64, 10000.0, "yarn", 8.0, original_length=4096)
    base = rotary.frequencies(64, 10000.0)[0]
    turns = 4096 * base / (2 * math.pi)
    assert np.allclose(y[turns > 40], base[turns > 40]) and np.allclose(y[turns < 0.8], base[turns < 0.8] / 8)
    assert np.all(y <= base) and np.all(y >= base / 8 * (1 - 1e-12)) and math.isclose(m, 0.1 * math.log(8) + 1)
    for bad in (dict(rot_dim=7), dict(rot_dim=8, base=0.0), dict(rot_dim=8, scaling="yarn"), dict(rot_dim=8, scaling="x")):
        with pytest.raises(ValueError):
            rotary.frequencies(**bad)


def test_table():
    import torch
    from unpermute_route_hist_gb300 import rotary
    f = rotary.rope_freqs(8, 100.0, sections=(1, 3), device="cpu")
    assert f.steps.dtype == torch.int64 and f.axes == 2 and list(f.c_sections) == [1, 3]
    inv = rotary.frequencies(8, 100.0)[0]
    for s, w in zip(f.steps.tolist(), inv):
        assert abs((s % 2 ** 64) / 2.0 ** 64 - w / (2 * math.pi)) < 2.0 ** -53
    with pytest.raises(ValueError):
        rotary.rope_freqs(8, sections=(1, 2), device="cpu")
