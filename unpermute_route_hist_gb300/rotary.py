"""Frequencies of rotary positions: the table gg_rope takes, from a head's rotated
width, the base and a scaling for contexts longer than the trained one.

Pair i of rot_dim / 2 turns by base^(-2i / rot_dim) radians a position.  Scalings:

  linear  positions are divided by factor (position interpolation)
  ntk     the base grows by factor^(rot / (rot - 2)): the slowest pair stretches by
          factor, the fastest keeps its speed
  yarn    pairs that turn more than beta_fast times over original_length keep their
          speed, those under beta_slow are interpolated by factor, a linear ramp over
          the pair index between; the result is scaled by 0.1 ln(factor) + 1 (by 1 for
          a factor up to 1)

The table is computed in 64 bits and held as fractions of a turn in units of 2^-64,
so the kernel reduces pos * f modulo one turn exactly.
"""
from __future__ import annotations

import ctypes
import dataclasses
import math

import numpy as np
import torch


@dataclasses.dataclass(frozen=True)
class RopeFreqs:
    steps: torch.Tensor             # [rot_dim / 2] int64, turns a position in units of 2^-64
    rot_dim: int
    attention_scale: float          # factor on the turned elements
    sections: tuple | None = None   # pairs of each position axis, or None (one axis)

    def __post_init__(self):
        if self.rot_dim < 0 or self.rot_dim % 2:
            raise ValueError("rot_dim must be even and not negative")
        s = self.steps
        if s.dtype is not torch.int64 or s.shape != (self.rot_dim // 2,) or not s.is_contiguous():
            raise ValueError("steps must be %d contiguous int64, got %s of %s" % (self.rot_dim // 2, tuple(s.shape), s.dtype))
        if self.sections is not None and (min(self.sections, default=-1) < 0 or sum(self.sections) != self.rot_dim // 2):
            raise ValueError("sections must be pair counts that sum to rot_dim / 2")
        # what a call passes on, made once
        axes = 1 if self.sections is None else len(self.sections)
        object.__setattr__(self, "axes", axes)
        object.__setattr__(self, "c_sections", (ctypes.c_int32 * axes)(*self.sections) if axes > 1 else None)


def frequencies(rot_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                original_length: int | None = None, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(radians a position of each pair [rot_dim / 2] float64, attention scale)."""
    if rot_dim < 0 or rot_dim % 2:
        raise ValueError("rot_dim must be even and not negative")
    if not (0 < base < math.inf and 0 < factor < math.inf):
        raise ValueError("base and factor must be positive and finite")
    if scaling == "ntk" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    pairs = np.arange(rot_dim // 2, dtype=np.float64)
    inv = base ** (-2.0 * pairs / max(rot_dim, 1))
    if scaling in (None, "ntk"):
        return inv, 1.0
    if scaling == "linear":
        return inv / factor, 1.0
    if scaling == "yarn":
        if not original_length or original_length < 0:
            raise ValueError("yarn needs original_length")
        if base <= 1 or not (beta_fast > 0 and beta_slow > 0):
            raise ValueError("yarn needs a base above 1 and positive betas")

        def pair_of(turns):  # pair index that turns this often over the original length
            return rot_dim * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))

        low = max(math.floor(pair_of(beta_fast)), 0)
        high = min(math.ceil(pair_of(beta_slow)), rot_dim - 1)
        ramp = np.clip((pairs - low) / max(high - low, 1e-3), 0.0, 1.0)
        return inv * (1.0 - ramp) + inv / factor * ramp, 0.1 * math.log(max(factor, 1.0)) + 1.0
    raise ValueError("unknown scaling %r" % (scaling,))


def rope_freqs(rot_dim: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
               original_length: int | None = None, beta_fast: float = 32.0, beta_slow: float = 1.0, sections=None,
               device="cuda") -> RopeFreqs:
    """The table for rope and rope_bwd.  sections: pairs of each position axis (sum
    rot_dim / 2), for positions [axes, T]."""
    if sections is not None:
        sections = tuple(int(s) for s in sections)
    inv, m = frequencies(rot_dim, base, scaling, factor, original_length, beta_fast, beta_slow)
    steps = [int(math.ldexp(float(f) / (2 * math.pi), 64)) & (2 ** 64 - 1) for f in inv]
    table = torch.from_numpy(np.array(steps, dtype=np.uint64).view(np.int64).copy())
    return RopeFreqs(table.to(device), rot_dim, float(m), sections)
