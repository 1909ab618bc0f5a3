"""Binding of the decode step's other entry points (include/swiglu.h has the
contracts), through the same native module as the paged-cache calls: norms of
heads with the position rotation, verification of drafted tokens, and products
with 4-bit weights.

    # a layer: q, k, v are slices of the fused projection's output
    q = swiglu_head_rotate_write(q, k, v, plan.positions, inv_freq, plan.slots,
                                 k_cache, v_cache, q_weight=qw, k_weight=kw)
    out = swiglu_mlp_forward_q4(x, Q1, S1, Q2, S2, Q3, S3)
    # a step: target is the softmax of its logits
    held = swiglu_verify_drafts(tokens, plan.query_start, target, parents=parents,
                                uniform=torch.rand(T, device="cuda"))
    ctx_lens = swiglu_cache_accept(k_caches, v_caches, block_table, ctx_lens,
                                   held.paths, held.path_lens)
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import cache, load_library
from .cache import _native, _on


def swiglu_head_rotate(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor,
                       inv_freq: torch.Tensor = None, q_weight: torch.Tensor = None,
                       k_weight: torch.Tensor = None, eps: float = 1e-6,
                       interleaved: bool = False, q_out: torch.Tensor = None,
                       k_out: torch.Tensor = None, stream=None):
    """(q, k) [tokens, heads, head size] BF16 (strided views allowed), each head
    divided by its root mean square and multiplied by its weight [head size]
    (None: left as it is), its first 2 * len(inv_freq) values then rotated by
    positions [tokens] int32 times inv_freq FP32 (None: not at all), in pairs
    (i, i + len(inv_freq)), or (2i, 2i + 1) if `interleaved`. `q_out` and `k_out`
    may be q and k themselves; by default they are new and contiguous."""
    f = (cache._binding or _native()).rotate
    if (q_out is None or k_out is None) and stream is not None:
        return _on(stream, f, q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved,
                   q_out, k_out, None)
    return f(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, q_out, k_out, stream)


def swiglu_head_rotate_write(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                             positions: torch.Tensor, inv_freq: torch.Tensor, slots: torch.Tensor,
                             k_cache: torch.Tensor, v_cache: torch.Tensor,
                             q_weight: torch.Tensor = None, k_weight: torch.Tensor = None,
                             eps: float = 1e-6, interleaved: bool = False,
                             q_out: torch.Tensor = None, stream=None) -> torch.Tensor:
    """swiglu_head_rotate whose keys go to their slots of the cache, and the values as
    they are beside them (swiglu_cache_write's slots and caches), in one launch.
    Returns q, rotated."""
    f = (cache._binding or _native()).rotate_write
    if q_out is None and stream is not None:
        return _on(stream, f, q, k, v, positions, inv_freq, slots, k_cache, v_cache, q_weight,
                   k_weight, eps, interleaved, None, None)
    return f(q, k, v, positions, inv_freq, slots, k_cache, v_cache, q_weight, k_weight, eps,
             interleaved, q_out, stream)


class Verified(NamedTuple):
    """What swiglu_verify_drafts finds; pass it as `out` to reuse its buffers (None in one's
    place: a new one)."""
    paths: torch.Tensor          # [R, width] int32: places of the tokens that hold, then -1
    path_lens: torch.Tensor      # [R] int32
    next_tokens: torch.Tensor    # [R] int32: the token that follows


def swiglu_verify_drafts(tokens: torch.Tensor, query_start: torch.Tensor, target: torch.Tensor,
                         parents: torch.Tensor = None, draft: torch.Tensor = None,
                         uniform: torch.Tensor = None, width: int = None, out: Verified = None,
                         stream=None) -> Verified:
    """Which of a step's `tokens` [T] int32 hold under the target, and what follows them.
    `target` [T, vocabulary] FP32 or BF16: row t is the distribution of the token
    after token t; `draft`, of the same type, what the tokens whose parent is t were drawn from
    (None: they were not drawn); `uniform` [T] FP32 in [0, 1): one random number a token.
    Or `target` [T] int32: the tokens that follow greedily (no draft, no uniform).
    `parents` [R, width] as for swiglu_cache_plan; chains (None) need `width`, the most
    tokens a request has."""
    f = (cache._binding or _native()).verify
    given = (None, None, None) if out is None else tuple(out)
    if stream is not None and any(t is None for t in given):
        return Verified(*_on(stream, f, tokens, query_start, target, parents, draft, uniform, width,
                             *given, None))
    return Verified(*f(tokens, query_start, target, parents, draft, uniform, width, *given, stream))


def swiglu_up_q4_workspace_bytes(M: int, N: int, K: int, group: int = 128) -> int:
    return int(load_library().swiglu_up_q4_workspace_bytes(int(M), int(N), int(K), int(group)))


def swiglu_down_q4_workspace_bytes(M: int, N: int, K: int, group: int = 128) -> int:
    return int(load_library().swiglu_down_q4_workspace_bytes(int(M), int(N), int(K), int(group)))


def swiglu_mlp_q4_workspace_bytes(M: int, N: int, K: int, group: int = 128) -> int:
    return int(load_library().swiglu_mlp_q4_workspace_bytes(int(M), int(N), int(K), int(group)))


def swiglu_up_forward_q4(A: torch.Tensor, Q1: torch.Tensor, S1: torch.Tensor, Q2: torch.Tensor,
                         S2: torch.Tensor, group: int = 128, Y: torch.Tensor = None,
                         workspace: torch.Tensor = None, stream=None) -> torch.Tensor:
    """Y[M, N] = SiLU(A W1^T) (.) (A W2^T) from A [M, K] BF16 and weights of 4-bit codes
    Q [N, K / 2] uint8 (low four bits: the even k) with scales S [ceil(K / group), N]
    BF16: W[n, k] = (code - 8) * S[k / group, n]. `workspace`: by default a new one, where
    one is used (swiglu_up_q4_workspace_bytes)."""
    f = (cache._binding or _native()).up_q4
    if stream is not None:
        return _on(stream, f, A, Q1, S1, Q2, S2, group, Y, workspace, None)
    return f(A, Q1, S1, Q2, S2, group, Y, workspace, None)


def swiglu_down_forward_q4(Y: torch.Tensor, Q3: torch.Tensor, S3: torch.Tensor, group: int = 128,
                           out: torch.Tensor = None, workspace: torch.Tensor = None,
                           stream=None) -> torch.Tensor:
    """out[M, K] = Y W3^T from Y [M, N] BF16, codes Q3 [K, N / 2] and scales S3
    [ceil(N / group), K]: the down-projection, and any other plain product."""
    f = (cache._binding or _native()).down_q4
    if stream is not None:
        return _on(stream, f, Y, Q3, S3, group, out, workspace, None)
    return f(Y, Q3, S3, group, out, workspace, None)


def swiglu_mlp_forward_q4(A: torch.Tensor, Q1: torch.Tensor, S1: torch.Tensor, Q2: torch.Tensor,
                          S2: torch.Tensor, Q3: torch.Tensor, S3: torch.Tensor, group: int = 128,
                          Y: torch.Tensor = None, out: torch.Tensor = None,
                          workspace: torch.Tensor = None, stream=None) -> torch.Tensor:
    """The whole gated MLP with 4-bit weights: swiglu_up_forward_q4 into Y [M, N]
    (caller's or a new buffer), then swiglu_down_forward_q4. Returns out [M, K]."""
    f = (cache._binding or _native()).mlp_q4
    if stream is not None:
        return _on(stream, f, A, Q1, S1, Q2, S2, Q3, S3, group, Y, out, workspace, None)
    return f(A, Q1, S1, Q2, S2, Q3, S3, group, Y, out, workspace, None)
