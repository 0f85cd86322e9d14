"""gg_rope refuses outputs whose own heads overlap (strides below the elements it writes): two
threads would write one element, and in place turn it twice.  No call here reaches the GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    from unpermute_route_hist_gb300 import _lib
    return _lib.load()


fake, other = ctypes.c_void_p(4096), ctypes.c_void_p(1 << 20)  # never dereferenced


def rope(lib, src, dst, tok, head, T=3, n=2, D=16, rot=8, of_k=False):
    none = (None, 0, 0, 0)
    x, y = (src, 64, 16, n), (dst, tok, head)
    steps = pos = fake
    (q, k) = (none, x) if of_k else (x, none)
    (oq, ok) = ((None, 0, 0), y) if of_k else (y, (None, 0, 0))
    return lib.gg_rope(q[0], q[1], q[2], q[3], k[0], k[1], k[2], k[3], *oq, *ok, pos, 1, None, steps, 1.0, T, D, rot, 0, 0,
                       0, None)


@pytest.mark.parametrize("of_k", [False, True])
@pytest.mark.parametrize("tok,head", [(0, 16), (64, 0), (8, 64), (64, 15)])
def test_overlapping_outputs(lib, tok, head, of_k):
    from unpermute_route_hist_gb300 import _lib
    assert rope(lib, fake, other, tok, head, of_k=of_k) == _lib.GG_ERR_INVALID_ARG


def test_overlapping_in_place(lib):
    """In place the rotated elements alone are written: strides may be as low as their number."""
    from unpermute_route_hist_gb300 import _lib

    def place(tok, head):
        return lib.gg_rope(fake, tok, head, 2, None, 0, 0, 0, fake, tok, head, None, 0, 0, fake, 1, None, fake, 1.0, 3, 16,
                           8, 0, 0, 0, None)

    assert place(0, 16) == place(64, 0) == place(7, 64) == place(64, 7) == _lib.GG_ERR_INVALID_ARG
