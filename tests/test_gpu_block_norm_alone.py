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
