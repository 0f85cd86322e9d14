"""Frequency tables at the ends of their arguments' ranges (host only)."""
import math

import numpy as np
import pytest


@pytest.mark.parametrize("factor", [1.0, 0.5, 1e-3, 1e-6])
def test_yarn_does_not_scale_down_for_factors_up_to_one(factor):
    """A context no longer than the trained one: the attention factor stays 1 (0.1 ln(factor) + 1
    would go below it, and below zero from e^-10 on)."""
    from unpermute_route_hist_gb300 import rotary
    inv, m = rotary.frequencies(64, 10000.0, "yarn", factor, original_length=4096)
    assert m == 1.0
    base = rotary.frequencies(64, 10000.0)[0]
    assert np.all(inv >= base * (1 - 1e-12)) and np.all(inv <= base / factor * (1 + 1e-12))


def test_yarn_attention_factor_above_one():
    from unpermute_route_hist_gb300 import rotary
    for factor in (1.0 + 1e-9, 2.0, 32.0):
        m = rotary.frequencies(64, 10000.0, "yarn", factor, original_length=4096)[1]
        assert math.isclose(m, 0.1 * math.log(factor) + 1.0, rel_tol=1e-15)


@pytest.mark.parametrize("bad", [
    dict(base=float("nan")), dict(base=float("inf")), dict(scaling="linear", factor=float("nan")),
    dict(scaling="linear", factor=float("inf")), dict(scaling="yarn", factor=float("inf"), original_length=4096),
    dict(scaling="yarn", base=1.0, factor=4.0, original_length=4096),
    dict(scaling="yarn", base=0.5, factor=4.0, original_length=4096),
    dict(scaling="yarn", factor=4.0, original_length=-4096),
    dict(scaling="yarn", factor=4.0, original_length=4096, beta_fast=0.0),
    dict(scaling="yarn", factor=4.0, original_length=4096, beta_slow=-1.0),
])
def test_refuses_what_gives_no_table(bad):
    """Not finite, or a logarithm of nothing: a ValueError that says so, no table of NaN or zeros."""
    from unpermute_route_hist_gb300 import rotary
    with pytest.raises(ValueError, match="must|needs"):
        rotary.rope_freqs(64, device="cpu", **bad)


def test_a_base_below_one_still_gives_a_table():
    from unpermute_route_hist_gb300 import rotary
    f = rotary.rope_freqs(8, 0.5, device="cpu")
    for s, p in zip(f.steps.tolist(), range(4)):
        assert abs((s % 2 ** 64) / 2.0 ** 64 - (0.5 ** (-p / 4) / (2 * math.pi)) % 1.0) < 2.0 ** -52


def test_a_hand_made_table_is_checked():
    """The kernel reads rot_dim / 2 steps of 64 bits: a table that holds fewer, or another type, is
    refused where it is made."""
    import torch
    from unpermute_route_hist_gb300.rotary import RopeFreqs
    steps = torch.arange(4, dtype=torch.int64)
    assert RopeFreqs(steps, 8, 1.0).axes == 1 and RopeFreqs(steps, 8, 1.0, (1, 3)).axes == 2
    assert RopeFreqs(steps[:0], 0, 1.0).rot_dim == 0
    for bad in ((steps[:3], 8), (steps, 6), (steps.to(torch.int32), 8), (steps.double(), 8), (steps.view(2, 2), 8),
                (torch.arange(8)[::2], 8), (steps, 7), (steps, -8)):
        with pytest.raises(ValueError):
            RopeFreqs(*bad, 1.0)
    for sections in ((1, 2), (-1, 5), ()):
        with pytest.raises(ValueError):
            RopeFreqs(steps, 8, 1.0, sections)
