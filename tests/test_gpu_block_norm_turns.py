"""Norms around a block with more tokens than CTAs (152 SMs, up to 24 CTAs each), so that every CTA takes several in turn:
its ring's stages are filled again and its column sums grow.  Bounds as in test_gpu_block_norm."""
import numpy as np
import pytest
import torch

import act8_ref as ref
import unpermute_route_hist_gb300 as gg
from gpu_util import dev, status_of, status_tensor
from test_gpu_block_norm import STREAMS, Inputs, U, check_backward, check_forward, close, run_backward, run_forward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


# two or three rows a token: 912 CTAs for 2048 columns, 3648 for 256, 456 for 4096, 152 for 8192
# (and their rows' odd neighbours); more: 608, 2432, 304, 152
@pytest.mark.parametrize("stream", STREAMS)
@pytest.mark.parametrize("T,K,topk", [(1831, 2048, 2), (7301, 256, 2), (923, 4096, 3), (311, 8192, 2), (1001, 2056, 3),
                                      (1301, 2048, 8), (5003, 136, 8), (635, 4096, 8), (159, 8192, 64), (2501, 264, 64)])
def test_combines(T, K, topk, stream):
    i = Inputs(T, K, stream, topk, topk=topk)
    st = status_tensor()
    got = run_forward(i, keep="bf16", status=st)
    assert status_of(st) == 0
    y, ysize = check_forward(i, got)
    close(got[2], y, ysize, (topk + 2) * U, "y")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("stream", STREAMS)
@pytest.mark.parametrize("T,K,topk", [(1831, 2048, 2), (923, 4104, 3), (311, 8192, 2), (7301, 264, 2), (1301, 2056, 8),
                                      (635, 4096, 8), (2501, 136, 33), (90, 8456, 3)])
def test_what_is_kept_of_a_sum(T, K, topk, stream, fmt):
    """Whole-number rows and weights: the sums are exact in fp32, so what is kept is the definition's."""
    g = torch.Generator().manual_seed(T)
    Y = torch.randint(-8, 9, (T * topk, K), generator=g)
    Y = (Y * 2 ** torch.randint(0, 5, (T * topk, 1), generator=g)).bfloat16()
    w = torch.randint(-3, 4, (T, topk), generator=g).float()
    m = torch.randperm(T * topk, generator=g).to(torch.int32)
    v = torch.ones(K, device=dev())
    kept = gg.block_norm(torch.zeros(T, K, dtype=stream, device=dev()), Y.to(dev()), w_post=v, w_pre=v, topk=topk,
                         row_id_map=m.to(dev()), topk_w=w.to(dev()), keep=fmt)[2]
    y = torch.einsum("tj,tjk->tk", w, Y.float()[m.long()].view(T, topk, K))
    assert float(y.abs().max()) < 2 ** 24
    packed = gg.act8_pack(y.to(dev()), fmt)
    nb = -(-K // 32)
    # (e4m3 has two zeros, and a sum of 0 may be either)
    assert torch.equal(kept.scales[:, :nb], packed.scales[:, :nb])
    table = torch.from_numpy(ref.TABLE[fmt]).to(dev())
    assert torch.equal(table[kept.codes.long()], table[packed.codes.long()])
    few = [0, T // 2, T - 1]
    c, s = ref.pack(y[few].double().numpy(), fmt)
    assert np.array_equal(kept.scales[few].cpu().numpy()[:, :nb], s)
    assert np.array_equal(ref.TABLE[fmt][kept.codes[few].cpu().numpy()], ref.TABLE[fmt][c])


# 304 CTAs for 4096 columns, 152 for 8192, 608 for 2048, 2432 for 512 and less
@pytest.mark.parametrize("kind", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("stream", STREAMS)
@pytest.mark.parametrize("T,K", [(919, 4096), (457, 8192), (1301, 2048), (5003, 512), (920, 4088), (331, 8184)])
def test_backward(T, K, stream, kind):
    i = Inputs(T, K, stream, T + K)
    if kind == "bf16":
        kept, y = i.y.to(dev()), i.y.double()
    else:
        kept = gg.act8_pack(i.y.to(dev()), kind)
        y = torch.from_numpy(ref.unpack(*ref.pack(i.y.double().numpy(), kind), K, kind))
    check_backward(i, y, run_backward(i, kept))
