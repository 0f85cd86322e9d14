"""Rotary positions on heads whose elements lie past 2^31 of their tensor, on a strided view:
63 of 64 heads, turned in place, give the bits of the same rows by themselves, and the head
between one token's and the next stays as it was.  (test_gpu_rope.py defines
test_offsets_past_32_bits twice, and only its second, of a packed projection, is collected.)"""
import pytest
import torch

from gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gg():
    import __graft_entry__ as g
    g.build()
    import unpermute_route_hist_gb300 as gg
    return gg


def test_strided_heads_past_2_31_elements(gg):
    T, H, D = 270000, 64, 128
    freqs = gg.rope_freqs(D, device=dev())
    pos = torch.arange(T, dtype=torch.int32, device=dev())
    buf = torch.empty(T, H, D, dtype=torch.bfloat16, device=dev()).normal_()
    for step in (gg.rope, gg.rope_bwd):
        want, _ = step(buf[-5:, :H - 1].contiguous(), None, pos[-5:].clone(), freqs)
        kept = buf[:, H - 1].clone()
        q = buf[:, :H - 1]
        step(q, None, pos, freqs, out_q=q)
        assert torch.equal(q[-5:], want) and torch.equal(buf[:, H - 1], kept)
    del buf, q, kept
    torch.cuda.empty_cache()


def test_one_token_or_one_head_of_any_stride(gg):
    """A single token's or head's stride does not matter: nothing overlaps."""
    freqs = gg.rope_freqs(16, device=dev())
    for T, H in ((1, 4), (5, 1), (1, 1)):
        x = torch.randn(T, H, 16, dtype=torch.bfloat16, device=dev())
        pos = torch.arange(1, T + 1, dtype=torch.int32, device=dev())
        want, _ = gg.rope(x, None, pos, freqs)
        y = torch.zeros(T, H, 16, dtype=torch.bfloat16, device=dev())
        out = y.as_strided((T, H, 16), (0 if T == 1 else H * 16, 0 if H == 1 else 16, 1))
        got, _ = gg.rope(x, None, pos, freqs, out_q=out)
        assert torch.equal(got, want)
    x = torch.randn(3, 1, 16, dtype=torch.bfloat16, device=dev()).expand(3, 4, 16)
    with pytest.raises(gg.GGError):
        gg.rope(x, None, torch.zeros(3, dtype=torch.int32, device=dev()), freqs, out_q=x)  # four heads in one place
