"""gg_forward_swiglu_act8 reads the experts' sizes while it writes: outputs over them, or over the slots, are refused."""
import pytest

from test_abi_act8_norm import INVALID, P


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    from unpermute_route_hist_gb300 import _lib
    return _lib.load()


def test_outputs_over_sizes_and_slots(lib):
    # [16, 64] codes (1024 bytes), [16, 4] scales, [16, 32] bf16 activations; 4 sizes, 16 slots
    ok = dict(X=P, W=2 * P, m=3 * P, g=None, px=0, codes=4 * P, scales=5 * P, A=6 * P)

    def call(**kw):
        a = {**ok, **kw}
        return lib.gg_forward_swiglu_act8(a["X"], a["W"], a["m"], a["g"], 8, 2, 4, 64, 64, a["px"], 0, a["codes"],
                                          a["scales"], a["A"], None, None)

    for bad in (dict(m=4 * P), dict(m=4 * P + 1020), dict(m=5 * P - 12), dict(m=6 * P + 1020), dict(codes=3 * P),
                dict(g=4 * P, px=1), dict(g=5 * P + 60, px=1), dict(g=6 * P - 60, px=1), dict(g=6 * P)):
        assert call(**bad) == INVALID, bad
