"""The norm of the stream alone, where h' is h whatever the residual's scale: its two directions, called with the
same arguments, against autograd in 64 bits.  Bounds as those of rows with a block: half a step of the output's type and
K / 16 + 32 fp32 steps of the magnitudes that are added, a column's T more."""
import pytest
import torch

import unpermute_route_hist_gb300 as gg
from gpu_util import dev
from test_gpu_block_norm import STREAMS, U, close, steps

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


@pytest.mark.parametrize("stream", STREAMS)
@pytest.mark.parametrize("scale", [0.5, -2.0, 0.0])
@pytest.mark.parametrize("T,K", [(1, 8), (50, 264), (40, 4096), (90, 8328)])
def test_a_scale_does_not_count(T, K, scale, stream):
    g = torch.Generator().manual_seed(T + K)
    rnd = lambda: torch.randn(T, K, generator=g)
    h, dh, dx, w = rnd().to(stream), rnd().to(stream), rnd().bfloat16(), torch.rand(K, generator=g) + 0.5
    on = lambda t: t.to(dev())
    out, x, kept = gg.block_norm(on(h), w_pre=on(w), res_scale=scale, eps=EPS)
    hv, wv = h.double().requires_grad_(), w.double().requires_grad_()
    want = hv / torch.sqrt((hv * hv).mean(1, keepdim=True) + EPS) * wv
    close(x, want.detach(), want.detach().abs(), steps(K), "x")
    assert kept is None and torch.equal(out.cpu(), h)
    ((hv * dh.double()).sum() + (want * dx.double()).sum()).backward()
    got = gg.block_norm_bwd(on(dh), on(dx), on(h), w_pre=on(w), res_scale=scale, eps=EPS)
    hd, r = h.double(), 1 / torch.sqrt((h.double() ** 2).mean(1, keepdim=True) + EPS)
    wd = (dx.double() * w.double()).abs()
    size = dh.double().abs() + r * (wd + (hd * r).abs() * (wd * (hd * r).abs()).mean(1, keepdim=True))
    close(got[0], hv.grad, 4 * size, steps(K), "dh")
    close(got[3], wv.grad, 8 * (dx.double() * hd * r).abs().sum(0), steps(K) + T * U, "dw_pre")
    assert got[1] is None and got[2] is None and got[4] is None and got[5] is None


@pytest.mark.parametrize("stream", STREAMS)
def test_rows_past_the_squares_range(stream):
    """Rows of 2^70, whose squares fp32 does not hold: normed to zeros, the zero gradient through the norm, and no
    trace in other tokens or in the weights' gradients."""
    T, K = 9, 520
    g = torch.Generator().manual_seed(4)
    on = lambda t: t.to(dev())
    h, y = torch.randn(T, K, generator=g).to(stream), torch.randn(T, K, generator=g).bfloat16()
    dh, dx = torch.randn(T, K, generator=g).to(stream), torch.randn(T, K, generator=g).bfloat16()
    v = dict(w_post=on(torch.rand(K, generator=g)), w_pre=on(torch.rand(K, generator=g)))
    h[3], y[6] = 2.0 ** 70, 2.0 ** 70
    h2, x2, _ = gg.block_norm(on(h), on(y), **v, res_scale=0.5)
    assert not x2[3].any() and torch.equal(h2[6].float().cpu(), 0.5 * h[6].float())
    got = gg.block_norm_bwd(on(dh), on(dx), on(h), on(y), **v, res_scale=0.5)
    want_h = (0.5 * dh[3].float()).to(stream)
    assert torch.equal(got[0][3].cpu(), want_h) and not got[1][6].any()
    rest = [t for t in range(T) if t not in (3, 6)]
    few = gg.block_norm_bwd(on(dh[rest]), on(dx[rest]), on(h[rest]), on(y[rest]), **v, res_scale=0.5)
    assert torch.equal(got[0][rest], few[0]) and torch.equal(got[1][rest], few[1])
    # the sums, without the norm that is lost: token 3 still has its y, token 6 its h'
    one = [gg.block_norm_bwd(on(dh[t:t + 1]), on(dx[t:t + 1]), on(h[t:t + 1]), on(y[t:t + 1]), **v, res_scale=0.5)
           for t in range(T)]
    assert not one[6][2].any() and not one[3][3].any()
    for k in (2, 3):
        parts = torch.stack([o[k] for o in one]).double()
        assert float((got[k].double() - parts.sum(0)).abs().max()) <= T * U * float(parts.abs().sum(0).max())
