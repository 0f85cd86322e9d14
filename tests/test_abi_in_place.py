"""An output in place stands for its own input alone: what else it would write over is refused.  Host checks only
(a call that passes them would launch, and none here does)."""
import pytest

from test_abi_act8_norm import INVALID, P, UNSUPPORTED, _bwd, _norm

H = 4 * 64 * 2  # bytes of a [4, 64] bf16 tensor, as the calls' are; a row is 128


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    from unpermute_route_hist_gb300 import _lib
    return _lib.load()


def test_norm_in_place_over_another_input(lib):
    Q = 10 * P
    for bad in (dict(Y=Q, map=11 * P),                       # expert rows that other tokens' CTAs read through the map
                dict(Y=Q, topk=2), dict(Y=Q, topk=2, w=11 * P, map=12 * P),
                dict(Y=Q + 128), dict(Y=Q - 128),            # the same buffer, a row on
                dict(Y=Q, dt=2),                             # rows of another length at the same address
                dict(post=Q + 16), dict(pre=Q), dict(gate=Q + H - 16), dict(tg=Q), dict(w=Q + 4), dict(map=Q + 8)):
        assert _norm(lib, **{**dict(h=Q, oh=Q), **bad}) == INVALID, bad
    # the refusal that comes behind the overlaps' leaves the call itself unlaunched
    for out in (dict(ox=Q), dict(oy=Q), dict(codes=Q, scales=5 * P), dict(codes=5 * P, scales=Q)):
        assert _norm(lib, h=Q, oh=Q, **out) == INVALID, out


def test_norm_bwd_in_place_over_another_input(lib):
    Q = 10 * P
    for bad in (dict(h=Q + 128), dict(h=Q - 128), dict(dx=Q + 128), dict(y=Q + 256), dict(dt=2, h=20 * P, dx=Q),
                dict(dt=2, y=Q), dict(y=None, codes=Q, scales=20 * P), dict(y=None, codes=20 * P, scales=Q + 4),
                dict(post=Q), dict(pre=Q + 16), dict(gate=Q + H - 16), dict(tg=Q)):
        assert _bwd(lib, **{**dict(dh=Q, odh=Q), **bad}) == INVALID, bad
    for out in (dict(dy=Q), dict(dpre=Q + 16), dict(dpost=Q), dict(dgate=Q), dict(tg=30 * P, dtg=Q), dict(ws=Q)):
        assert _bwd(lib, dh=Q, odh=Q, **out) == INVALID, out
    assert _bwd(lib, dh=Q + 8, odh=Q + 8) == UNSUPPORTED
