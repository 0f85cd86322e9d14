"""Rotary positions: gg_rope forward and backward against the formula in float64.

Bounds (derived before any run): cos and sin are fp32 values of an angle reduced
exactly (a few ulp, 2^-22 of the pair's magnitude with the two products and the
sum), then one rounding to the output type: 2^-8 (bf16), 2^-11 (fp16), 2^-23
(fp32) of the value; fp16 values under its normal range round to 2^-25."""
import math

import numpy as np
import pytest
import torch

from gpu_util import dev

pytestmark = pytest.mark.gpu

ULP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -23}


@pytest.fixture(scope="module")
def gg():
    import __graft_entry__ as g
    g.build()
    import unpermute_route_hist_gb300 as gg
    return gg


def turned(x, pos, inv, m, interleaved, sections, backward):
    """(value, pair magnitude) of x [T, H, D] float64; pos [axes, T]."""
    rot = 2 * len(inv)
    axis = np.zeros(rot // 2, int) if sections is None else np.repeat(np.arange(len(sections)), sections)
    th = pos[axis].T.astype(np.float64) * inv
    th = -th if backward else th
    c, s = m * np.cos(th)[:, None], m * np.sin(th)[:, None]
    first = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    second = first + (1 if interleaved else rot // 2)
    y, mag = x.copy(), np.zeros_like(x)
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., second] * c + x[..., first] * s
    mag[..., first] = mag[..., second] = m * (np.abs(x[..., first]) + np.abs(x[..., second]))
    return y, mag


# float64 reference of the angle: pos * inv in float64 is good to 2^-53 * 2^31 * 2^53... for
# positions up to 2^20 the product's error is below 2^-32 of a radian
CASES = [
    # T, Hq, Hk, D, rot, interleaved, dtype, scaling, sections
    (1, 1, 0, 2, 2, False, torch.float32, {}, None),
    (1, 32, 8, 128, 128, False, torch.bfloat16, {}, None),
    (5, 3, 1, 64, 64, True, torch.float16, {}, None),
    (37, 4, 2, 80, 20, True, torch.float16, dict(scaling="linear", factor=4.0), None),
    (64, 2, 2, 96, 34, False, torch.bfloat16, dict(scaling="ntk", factor=2.0), None),
    (257, 5, 1, 192, 64, True, torch.float32, dict(scaling="yarn", factor=32.0, original_length=4096), None),
    (300, 7, 3, 66, 66, False, torch.float32, {}, (9, 12, 12)),
    (129, 4, 4, 128, 96, False, torch.bfloat16, {}, (8, 0, 24, 16)),
    (1000, 2, 1, 13, 6, True, torch.bfloat16, {}, None),
    (700, 16, 4, 256, 256, True, torch.bfloat16, dict(scaling="yarn", factor=4.0, original_length=8192), (64, 64)),
    (50, 3, 0, 40, 0, False, torch.float16, {}, None),
]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,rot,interleaved,dtype,scaling,sections", CASES)
def test_rope(gg, T, Hq, Hk, D, rot, interleaved, dtype, scaling, sections, backward):
    from unpermute_route_hist_gb300 import rotary
    g = np.random.default_rng(T)
    freqs = gg.rope_freqs(rot, sections=sections, device=dev(), **scaling)
    inv, m = rotary.frequencies(rot, **scaling)
    axes = len(sections) if sections else 1
    pos = g.integers(0, 1 << 20, (axes, T)).astype(np.int32)
    pos[:, 0] = 0
    q = torch.from_numpy(g.standard_normal((T, Hq, D))).to(dtype).to(dev())
    k = torch.from_numpy(g.standard_normal((T, Hk, D))).to(dtype).to(dev()) if Hk else None
    p = torch.from_numpy(pos if sections else pos[0]).to(dev())
    fn = gg.rope_bwd if backward else gg.rope
    outs = fn(q, k, p, freqs, interleaved=interleaved)
    for x, y in zip((q, k), outs):
        if x is None:
            assert y is None
            continue
        x64 = x.double().cpu().numpy()
        ref, mag = turned(x64, pos, inv, m, interleaved, sections, backward)
        err = np.abs(y.double().cpu().numpy() - ref)
        bound = ULP[dtype] * np.abs(ref) + 2.0 ** -21 * mag + (2.0 ** -25 if dtype == torch.float16 else 0.0)
        bound[..., rot:] = 0.0  # the rest of the head is copied
        assert (err <= bound).all(), (err.max(), np.argwhere(err > bound)[0])
    # in place gives the same bits
    q2 = q.clone()
    k2 = None if k is None else k.clone()
    fn(q2, k2, p, freqs, interleaved=interleaved, out_q=q2, out_k=k2)
    assert torch.equal(q2, outs[0]) and (k is None or torch.equal(k2, outs[1]))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,off", [(128, 0), (128, 1), (30, 3), (36, 2)])
def test_strided_and_unaligned_heads(gg, D, off, interleaved):
    """q and k as views of a packed projection that starts `off` elements into its
    buffer; v between tokens stays as it was; k transposed (heads outermost)."""
    T, Hq, Hk, rot = 45, 4, 2, D - D % 4
    width = (Hq + 2 * Hk) * D
    buf = torch.randn(T * width + off, dtype=torch.bfloat16, device=dev())
    kt = torch.randn(Hk, T, D, dtype=torch.bfloat16, device=dev()).transpose(0, 1)
    qkv = buf[off:].view(T, width)
    q = qkv[:, :Hq * D].view(T, Hq, D)
    pos = torch.randint(-1000, 100000, (T,), dtype=torch.int32, device=dev())
    freqs = gg.rope_freqs(rot, device=dev())
    want = gg.rope(q.contiguous(), kt.contiguous(), pos, freqs, interleaved=interleaved)
    rest = qkv[:, Hq * D:].clone()
    gg.rope(q, kt, pos, freqs, interleaved=interleaved, out_q=q, out_k=kt)
    assert torch.equal(q, want[0]) and torch.equal(kt, want[1]) and torch.equal(qkv[:, Hq * D:], rest)


def test_positions_are_exact_at_any_size(gg):
    """Position p + n * period of a pair whose step divides the turn gives position p's
    bits, at both ends of the int32 range."""
    freqs = gg.rope_freqs(2, device=dev())
    freqs = type(freqs)(torch.tensor([1 << 48], dtype=torch.int64, device=dev()), 2, 1.0)  # 2^-16 turns
    q = torch.randn(1, 1, 2, dtype=torch.float32, device=dev()).expand(5, 1, 2).contiguous()
    pos = torch.tensor([77, 77 + (1 << 16), 77 + (1 << 30), 77 - (1 << 31), 77 - (1 << 16)], dtype=torch.int32,
                       device=dev())
    y, _ = gg.rope(q, None, pos, freqs)
    assert all(torch.equal(y[0], y[i]) for i in range(5))
    th = 2 * math.pi * 77 / 65536
    x = q[0, 0].double().cpu()
    assert abs(float(y[0, 0, 0]) - float(x[0] * math.cos(th) - x[1] * math.sin(th))) <= 2.0 ** -21 * float(x.abs().sum())


def test_backward_is_the_gradient(gg):
    """The map is linear: <dy, rope(x)> = <rope_bwd(dy), x> for any x and dy (fp32: the
    rounding of 2 T H D terms, 2^-20 of the sum of magnitudes), and differences of the
    forward along x give the same number."""
    T, H, D = 65, 3, 64
    freqs = gg.rope_freqs(48, device=dev(), scaling="yarn", factor=8.0, original_length=2048)
    pos = torch.randint(0, 50000, (T,), dtype=torch.int32, device=dev())
    x, dy = (torch.randn(T, H, D, device=dev()) for _ in range(2))
    y, _ = gg.rope(x, None, pos, freqs)
    dx, _ = gg.rope_bwd(dy, None, pos, freqs)
    lhs, rhs = float((dy.double() * y.double()).sum()), float((dx.double() * x.double()).sum())
    tol = 2.0 ** -20 * float((dy.double().abs() * y.double().abs()).sum() + (dx.double().abs() * x.double().abs()).sum())
    assert abs(lhs - rhs) <= tol
    h = torch.randn_like(x)
    up, dn = gg.rope(x + h, None, pos, freqs)[0], gg.rope(x - h, None, pos, freqs)[0]
    num = float((dy.double() * (up.double() - dn.double())).sum()) / 2
    tol += 2.0 ** -20 * float((dy.double().abs() * (up.double().abs() + dn.double().abs())).sum())
    assert abs(num - float((dx.double() * h.double()).sum())) <= tol


def test_infinities_stay_in_their_pair(gg):
    freqs = gg.rope_freqs(64, device=dev())
    pos = torch.arange(9, dtype=torch.int32, device=dev())
    q = torch.randn(9, 2, 64, dtype=torch.bfloat16, device=dev())
    want, _ = gg.rope(q, None, pos, freqs)
    q[4, 1, 5] = float("inf")
    got, _ = gg.rope(q, None, pos, freqs)
    same = torch.ones_like(want, dtype=torch.bool)
    same[4, 1, 5] = same[4, 1, 37] = False
    assert torch.equal(got[same], want[same]) and not torch.isfinite(got[4, 1, 5])


def test_offsets_past_32_bits(gg):
    """Heads whose elements lie past 2^31 of their tensor, in place on a strided view."""
    T, H, D = 270000, 64, 128
    buf = torch.randn(T, H, D, dtype=torch.bfloat16, device=dev())
    freqs = gg.rope_freqs(D, device=dev())
    pos = torch.arange(T, dtype=torch.int32, device=dev())
    want, _ = gg.rope(buf[-5:, :63].contiguous(), None, pos[-5:], freqs)
    keep = buf[-5:, 63].clone()
    q = buf[:, :63]
    gg.rope(q, None, pos, freqs, out_q=q)
    assert torch.equal(q[-5:], want) and torch.equal(buf[-5:, 63], keep)


def test_empty_and_refusals(gg):
    freqs = gg.rope_freqs(64, device=dev())
    pos = torch.zeros(4, dtype=torch.int32, device=dev())
    q = torch.randn(4, 2, 64, dtype=torch.bfloat16, device=dev())
    assert gg.rope(q[:0], None, pos[:0], freqs)[0].shape == (0, 2, 64)
    assert gg.rope(q[:, :0], q, pos, freqs)[0].shape == (4, 0, 64)
    with pytest.raises(ValueError):
        gg.rope(q[..., :32], None, pos, freqs)                      # narrower than the table
    with pytest.raises(ValueError):
        gg.rope(q, q.float(), pos, freqs)
    with pytest.raises(ValueError):
        gg.rope(q, None, pos[:3], freqs)
    with pytest.raises(TypeError):
        gg.rope(q, None, pos.long(), freqs)
    with pytest.raises(TypeError):
        gg.rope(q.double(), None, pos, freqs)
    with pytest.raises(ValueError):
        gg.rope(q.transpose(1, 2).contiguous().transpose(1, 2), None, pos, freqs)
    with pytest.raises(ValueError):
        gg.rope(q, None, pos, freqs, out_q=q[:, :1])
    with pytest.raises(ValueError):
        gg.rope(q, None, pos, gg.rope_freqs(64, device="cpu"))
    big = gg.rope_freqs(2048, device=dev())
    with pytest.raises(gg.GGError):
        gg.rope(torch.zeros(1, 1, 2048, dtype=torch.bfloat16, device=dev()), None, pos[:1], big)


def test_offsets_past_32_bits(gg):
    """The last heads of a packed projection of more than 2^31 elements, in place: the bits of
    the same rows by themselves, and nothing beside them changes."""
    T, width, H, D, last = 360000, 6144, 2, 128, 300
    buf = torch.zeros(T, width, dtype=torch.bfloat16, device=dev())
    buf[-last:] = torch.randn(last, width, device=dev())
    tail = buf[-last:].clone()
    heads = lambda x: x[:, width - H * D:].view(x.shape[0], H, D)
    pos, freqs = torch.arange(T, dtype=torch.int32, device=dev()), gg.rope_freqs(D, device=dev())
    for step in (gg.rope, gg.rope_bwd):
        step(heads(buf), None, pos, freqs, out_q=heads(buf))
        step(heads(tail), None, pos[-last:].clone(), freqs, out_q=heads(tail))
        assert torch.equal(buf[-last:], tail) and not buf[:last].any()
