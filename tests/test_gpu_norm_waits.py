"""The norms' exits behind a wait that runs out, without a fault: the diagnostic entry points leave out the copies of one
stage, the wait for them ends after its limit, and the CTAs that share the row leave with nothing of theirs under way.
Every other row is an ordinary call's, and the context stays usable."""
import pytest
import torch

import unpermute_route_hist_gb300 as gg
from gpu_util import dev, status_of, status_tensor
from unpermute_route_hist_gb300 import _lib

pytestmark = pytest.mark.gpu
UNUSED, KEPT = -7, 3.0


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    return _lib.load()


def rows(T, K, seed):
    g = torch.Generator(device=dev()).manual_seed(seed)
    return torch.randn(T, K, device=dev(), generator=g).bfloat16()


def check(record, status, groups, wide, T, withheld, outs, wants):
    """groups: CTAs, or clusters of two, that take rows in turn."""
    assert status_of(status) == _lib.GG_DEV_TIMEOUT
    n = groups * (2 if wide else 1)
    r = record.cpu().view(-1, 3)
    assert (r[n:] == UNUSED).all()
    at = withheld % groups
    left = {2 * at, 2 * at + 1} if wide else {at}
    assert set(r[:n, 0].nonzero().flatten().tolist()) == left
    assert not r[:n, 1].any(), "stages filled and not waited for: %s" % r[:n, 1].nonzero().flatten().tolist()
    assert not r[:n, 2].any(), "stages filled again too early: %s" % r[:n, 2].nonzero().flatten().tolist()
    t = torch.arange(T, device=dev())
    lost = (t % groups == at) & (t >= withheld)
    for got, want in zip(outs, wants):
        assert torch.equal(got[~lost], want[~lost]) and (got[lost] == KEPT).all()


# rows of one CTA (1216 of them), of two (76 clusters)
@pytest.mark.parametrize("T,K,groups", [(1216 * 4 + 7, 520, 1216), (76 * 6 + 5, 8456, 76)])
def test_backward(lib, T, K, groups):
    h, dx, y = (rows(T, K, s) for s in (1, 2, 3))
    w = torch.rand(K, device=dev()) + 0.5
    call = lambda: gg.block_norm_bwd(dx, dx, h, y, w_post=w, w_pre=w, want=(True, True, False))[:2]
    want = call()
    for turn in (0, 2):
        withheld = turn * groups + 10
        outs = [torch.full_like(h, KEPT) for _ in range(2)]
        record = torch.full((3 * 2432,), UNUSED, dtype=torch.int32, device=dev())
        status = status_tensor()
        rc = lib.gg_selftest_block_norm_bwd_wait(dx.data_ptr(), h.data_ptr(), y.data_ptr(), w.data_ptr(), T, K, withheld,
                                                 outs[0].data_ptr(), outs[1].data_ptr(), record.data_ptr(), status.data_ptr(),
                                                 torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        check(record, status, groups, K > 8192, T, withheld, outs, want)
    assert all(torch.equal(a, b) for a, b in zip(call(), want))


# several stages a token: 64 rows of 4104 columns (152 CTAs), 40 of 8456 (76 clusters)
@pytest.mark.parametrize("T,K,topk,groups", [(152 * 3 + 5, 4104, 64, 152), (76 * 3 + 5, 8456, 40, 76)])
def test_forward(lib, T, K, topk, groups):
    h, Y = rows(T, K, 1), rows(T * topk, K, 2)
    w = torch.rand(K, device=dev()) + 0.5
    call = lambda: gg.block_norm(h, Y, w_post=w, w_pre=w, topk=topk)[:2]
    want = call()
    for turn in (0, 1):
        withheld = turn * groups + 10
        outs = [torch.full_like(h, KEPT) for _ in range(2)]
        record = torch.full((3 * 2432,), UNUSED, dtype=torch.int32, device=dev())
        status = status_tensor()
        rc = lib.gg_selftest_block_norm_wait(h.data_ptr(), Y.data_ptr(), topk, w.data_ptr(), T, K, withheld, outs[0].data_ptr(),
                                             outs[1].data_ptr(), record.data_ptr(), status.data_ptr(),
                                             torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        check(record, status, groups, K > 8192, T, withheld, outs, want)
    assert all(torch.equal(a, b) for a, b in zip(call(), want))


def test_refusals(lib):
    assert lib.gg_selftest_block_norm_bwd_wait(None, None, None, None, 4, 64, 0, None, None, None, None, None) == \
        _lib.GG_ERR_INVALID_ARG
    assert lib.gg_selftest_block_norm_wait(None, None, 8, None, 4, 64, 0, None, None, None, None, None) == _lib.GG_ERR_INVALID_ARG
