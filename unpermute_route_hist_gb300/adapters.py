"""The query/key/value projection of an attention block with the low-rank adapters of
many requests beside it and rotary positions on its query and key heads: the two
operators chained as a model uses them, forward (training, prefill, decoding) and
backward.

One packed weight W [(n_q + 2 n_kv) * head_dim, hidden] gives q | k | v; each token's
row takes its own adapter (gg_lora_forward), then the q and k heads are turned in place
(gg_rope).  The backward turns the packed gradient's q and k heads back in place, then
gives dX and the adapters' gradients (gg_lora_backward); W is frozen.

Every step runs in libgg.so's kernels.  The plan of a batch's adapter ids
(api.lora_plan) is made once and serves every layer.
"""
from __future__ import annotations

import dataclasses

import torch

from . import api


@dataclasses.dataclass
class Saved:
    """What the backward needs of a forward: its input and its low-rank activations."""
    X: torch.Tensor
    U: torch.Tensor
    plan: api.LoraPlan
    positions: torch.Tensor


class AdaptedQKV:
    """W [(n_q + 2 n_kv) * head_dim, hidden], A [L, r, hidden], B [L, (n_q + 2 n_kv) *
    head_dim, r] bf16; scale [L] fp32 or None; freqs from rope_freqs, or None for a
    projection without positions."""

    def __init__(self, W, A, B, scale, n_q: int, n_kv: int, head_dim: int, freqs, interleaved: bool = False):
        if W.shape[0] != (n_q + 2 * n_kv) * head_dim:
            raise ValueError("W must have (n_q + 2 n_kv) * head_dim rows")
        if freqs is not None and freqs.rot_dim > head_dim:
            raise ValueError("freqs turn %d elements of a head of %d" % (freqs.rot_dim, head_dim))
        self.W, self.A, self.B, self.scale = W, A, B, scale
        self.n_q, self.n_kv, self.head_dim = n_q, n_kv, head_dim
        self.freqs, self.interleaved = freqs, interleaved

    def split(self, qkv):
        """q [T, n_q, D], k and v [T, n_kv, D]: views of the packed rows."""
        T, D = qkv.shape[0], self.head_dim
        heads = qkv.view(T, self.n_q + 2 * self.n_kv, D)
        return heads[:, :self.n_q], heads[:, self.n_q:self.n_q + self.n_kv], heads[:, self.n_q + self.n_kv:]

    def forward(self, X, plan, positions, *, out=None, status=None):
        """(q, k, v, saved) for X [T, hidden]: views of one packed tensor."""
        qkv, U = api.lora_forward(X, self.W, self.A, self.B, self.scale, plan, out=out, status=status)
        q, k, v = self.split(qkv)
        if self.freqs is not None:
            api.rope(q, k, positions, self.freqs, interleaved=self.interleaved, out_q=q, out_k=k)
        return q, k, v, Saved(X, U, plan, positions)

    def backward(self, dqkv, saved: Saved, *, want=(True, True, True), status=None):
        """(dX, dA, dB) from the packed gradient dqkv [T, (n_q + 2 n_kv) * head_dim] of
        q | k | v, whose q and k heads are turned back in place."""
        if self.freqs is not None:
            dq, dk, _ = self.split(dqkv)
            api.rope_bwd(dq, dk, saved.positions, self.freqs, interleaved=self.interleaved, out_q=dq, out_k=dk)
        return api.lora_backward(dqkv, saved.X, self.W, self.A, self.B, self.scale, saved.plan, saved.U, want=want,
                                 status=status)
