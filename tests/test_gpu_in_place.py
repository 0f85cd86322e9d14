"""What may lie at the address of an output in place gives the bits of a call with tensors of their own."""
import pytest
import torch

import unpermute_route_hist_gb300 as gg
from gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


@pytest.mark.parametrize("T,K", [(5, 40), (700, 2048), (200, 8456)])
def test_every_row_input_at_once(T, K):
    g = torch.Generator().manual_seed(T)
    t = torch.randn(T, K, generator=g).bfloat16().to(dev())
    v = dict(w_post=torch.rand(K, generator=g).to(dev()), w_pre=torch.rand(K, generator=g).to(dev()))
    w = torch.rand(T, 1, generator=g).to(dev())
    for more in ({}, dict(topk_w=w)):
        want = gg.block_norm(t, t, **v, **more)
        p = t.clone()
        got = gg.block_norm(p, p, **v, **more, out_h=p)
        assert got[0] is p and torch.equal(p, want[0]) and torch.equal(got[1], want[1])
    want = gg.block_norm_bwd(t, t, t, t, **v)
    p = t.clone()
    got = gg.block_norm_bwd(p, p, p, p, **v, out=p)
    assert got[0] is p
    for a, b in zip(got, want):
        assert a is b is None or torch.equal(a, b)


def test_expert_rows_in_place_are_refused():
    """The stream as a view of the rows that the combine gathers: other tokens' rows would be written over."""
    T, K = 6, 64
    Y = torch.zeros(2 * T, K, dtype=torch.bfloat16, device=dev())
    w = torch.ones(K, device=dev())
    m = torch.arange(T, dtype=torch.int32, device=dev())
    h = Y[:T]
    for rows, more in ((Y, dict(topk=2)), (h, dict(row_id_map=m)), (Y[1:T + 1], {})):
        with pytest.raises(gg.GGError):
            gg.block_norm(h, rows, w_pre=w, out_h=h, **more)
    with pytest.raises(gg.GGError):
        gg.block_norm_bwd(h, Y[T:], Y[1:T + 1], w_pre=w, out=h)
