"""Refusals of the norms' diagnostic entry points, before any CUDA work."""
import pytest

from test_abi_act8_norm import INVALID, P, UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    from unpermute_route_hist_gb300 import _lib
    return _lib.load()


def test_forward(lib):
    ok = dict(h=P, Y=2 * P, topk=4, w=3 * P, T=8, K=64, held=3, oh=4 * P, ox=5 * P, rec=6 * P, st=7 * P)

    def call(**kw):
        a = {**ok, **kw}
        return lib.gg_selftest_block_norm_wait(a["h"], a["Y"], a["topk"], a["w"], a["T"], a["K"], a["held"], a["oh"], a["ox"],
                                               a["rec"], a["st"], None)

    for bad in (dict(h=None), dict(Y=None), dict(w=None), dict(oh=None), dict(ox=None), dict(rec=None), dict(st=None),
                dict(topk=3), dict(held=-1), dict(held=8), dict(T=0), dict(K=-8), dict(oh=2 * P), dict(ox=4 * P)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(K=12), dict(K=16392), dict(topk=65), dict(rec=6 * P + 2), dict(st=7 * P + 1), dict(h=P + 8)):
        assert call(**bad) == UNSUPPORTED, bad


def test_backward(lib):
    ok = dict(dx=P, h=2 * P, y=3 * P, w=4 * P, T=8, K=64, held=3, odh=5 * P, dy=6 * P, rec=7 * P, st=8 * P)

    def call(**kw):
        a = {**ok, **kw}
        return lib.gg_selftest_block_norm_bwd_wait(a["dx"], a["h"], a["y"], a["w"], a["T"], a["K"], a["held"], a["odh"],
                                                   a["dy"], a["rec"], a["st"], None)

    for bad in (dict(dx=None), dict(h=None), dict(y=None), dict(w=None), dict(odh=None), dict(dy=None), dict(rec=None),
                dict(st=None), dict(held=-1), dict(held=8), dict(T=0), dict(K=-8), dict(odh=2 * P), dict(dy=5 * P)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(K=12), dict(K=16392), dict(rec=7 * P + 2), dict(st=8 * P + 1), dict(y=3 * P + 8)):
        assert call(**bad) == UNSUPPORTED, bad
