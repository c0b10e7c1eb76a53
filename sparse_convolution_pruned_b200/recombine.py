"""Temporal recombination of projected tokens, forward and backward (SV-TAD page, Key Design 3, with
learned projections): the queries and keys of two token streams are normed per head and rotated by
their tokens' coordinates, and every query row attends over the keys of its group.

    Yq, Yk = norm + rotation of Q, K        (svconv_qk_norm_rope_fwd, one launch)
    O      = cross-attention of Yq, Yk, V   (svconv_cross_attn_fwd)

``recombine_bwd`` runs the adjoints in turn.  Positions are the coords tables of the index build
((t, y, x) per token) or any int32 [n] / [n, axes]; the groups are CSR offsets over the rows, like
frame_off.  Marshalling only: every step runs in the library's kernels.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional, Sequence

import torch

from . import svconv


@dataclass
class Groups:
    """Which rows of the two streams belong together."""
    q_off: torch.Tensor    # [G + 1] int32
    kv_off: torch.Tensor   # [G + 1] int32
    max_q: int             # bounds on a group's rows
    max_kv: int


@dataclass
class Rotation:
    """Rotary frequencies, and which coordinate each pair of channels follows."""
    freq: torch.Tensor                 # [rot / 2] fp64, radians per unit of position
    axis_pairs: Sequence[int]          # pairs that follow each axis
    layout: str = "half"
    eps: float = 1e-6                  # of the norm


def axis_frequencies(pairs: Sequence[int], base: float = 10000.0, device="cuda") -> torch.Tensor:
    """base^(-i / n) for the n pairs of each axis, one axis after the other."""
    f = [base ** (-i / n) for n in pairs for i in range(n)]
    return torch.tensor(f, dtype=torch.float64, device=device)


@dataclass
class Saved:
    """What recombine_bwd needs of the forward pass."""
    Q: torch.Tensor
    K: torch.Tensor
    V: torch.Tensor
    pos_q: torch.Tensor
    pos_k: torch.Tensor
    wq: Optional[torch.Tensor]
    wk: Optional[torch.Tensor]
    Yq: torch.Tensor
    Yk: torch.Tensor
    O: torch.Tensor
    lse: torch.Tensor
    kv_keep: Optional[torch.Tensor]
    scale: Optional[float]


def recombine_fwd(Q, K, V, pos_q, pos_k, groups: Groups, rotation: Rotation, *, wq=None, wk=None, kv_keep=None,
                  scale: Optional[float] = None, status=None, stream=None):
    """Q [nq, Hq, d], K and V [nkv, Hkv, d] bf16 -> (O [nq, Hq, d] bf16, Saved).  O's rows of no group are left
    as they were allocated."""
    Yq, Yk = svconv.svconv_qk_norm_rope_fwd(Q, K, pos_q, pos_k, rotation.freq, wq=wq, wk=wk, eps=rotation.eps,
                                            layout=rotation.layout, axis_pairs=rotation.axis_pairs, stream=stream)
    O, lse = svconv.svconv_cross_attn_fwd(Yq, Yk, V, groups.q_off, groups.kv_off, max_q=groups.max_q,
                                          max_kv=groups.max_kv, scale=scale, kv_keep=kv_keep, status=status,
                                          stream=stream)
    return O, Saved(Q, K, V, pos_q, pos_k, wq, wk, Yq, Yk, O, lse, kv_keep, scale)


def recombine_bwd(dO, saved: Saved, groups: Groups, rotation: Rotation, *, status=None, stream=None):
    """(dQ, dK, dV bf16, dwq, dwk fp32 [d]) of recombine_fwd.  As long as what they hold is finite, rows of no group
    (a padded batch's) get zero gradients, and they and left-out keys add nothing to dwq and dwk."""
    with torch.cuda.stream(stream):
        grads = [torch.zeros_like(t, memory_format=torch.contiguous_format) for t in (saved.Yq, saved.Yk, saved.V)]
    if stream is not None:  # that stream's memory, which the caller may use on the current one
        for t in grads:
            t.record_stream(torch.cuda.current_stream(dO.device))
    dYq, dYk, dV = svconv.svconv_cross_attn_bwd(dO, saved.Yq, saved.Yk, saved.V, saved.O, saved.lse, groups.q_off,
                                                groups.kv_off, max_q=groups.max_q, max_kv=groups.max_kv,
                                                scale=saved.scale, kv_keep=saved.kv_keep, dQ=grads[0], dK=grads[1],
                                                dV=grads[2], status=status, stream=stream)
    dQ, dK, dwq, dwk = svconv.svconv_qk_norm_rope_bwd(
        dYq, dYk, saved.Q, saved.K, saved.pos_q, saved.pos_k, rotation.freq, wq=saved.wq, wk=saved.wk, eps=rotation.eps,
        layout=rotation.layout, axis_pairs=rotation.axis_pairs, dQ=dYq, dK=dYk, stream=stream)
    return dQ, dK, dV, dwq, dwk
