"""Binding of the paged-cache entry points: argument checks and marshalling
only, as in the package's __init__ (include/swiglu.h has the contracts), here
in a small native module (csrc/cache_binding.cpp) because the calls are short.

One step of a batch that verifies drafted tokens:

    plan = swiglu_cache_plan(ctx_lens, new_lens, pages_held, block_table,
                             free_pages, page_size, max_tokens, parents=parents)
    # per layer: q, k, v of the step's tokens (rotated by plan.positions)
    swiglu_cache_write(k, v, plan.slots, k_cache, v_cache)
    out = swiglu_tree_attention(q, k_cache, v_cache, block_table, ctx_lens,
                                plan.query_start, mask=plan.mask)
    # once the accepted path of every request is known, all layers at once
    ctx_lens = swiglu_cache_accept(k_caches, v_caches, block_table, ctx_lens,
                                   paths, path_lens)

Caches are [pages, kv heads, page size, head size] BF16 (swiglu_cache_accept
also takes [layers, ...]); lengths, tables and slots are int32, masks int64.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
from typing import NamedTuple, Optional

import torch

from . import SwigluError, load_library
from .build import BINDING_PATH, binding_needs

_binding = None


def _native():
    """The binding module (csrc/cache_binding.cpp), connected to the library;
    raises if either has not been built."""
    global _binding
    if _binding is None:
        lib = load_library()
        if not os.path.exists(BINDING_PATH):
            missing = binding_needs()
            raise RuntimeError("%s is not built%s; run `python -m gemm_swiglu_mlp_gb300.build`"
                               % (os.path.basename(BINDING_PATH),
                                  " (it needs %s)" % ", ".join(missing) if missing else ""))
        loader = importlib.machinery.ExtensionFileLoader("_cache_binding", BINDING_PATH)
        spec = importlib.util.spec_from_file_location("_cache_binding", BINDING_PATH, loader=loader)
        mod = importlib.util.module_from_spec(spec)
        loader.exec_module(mod)
        mod.connect(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.swiglu_cache_plan, lib.swiglu_cache_write,
            lib.swiglu_tree_attention_workspace_bytes, lib.swiglu_tree_attention,
            lib.swiglu_cache_accept)), SwigluError, _workspace)
        _binding = mod
    return _binding


def _workspace(index: int, nbytes: int, stream) -> torch.Tensor:
    """A new attention workspace, allocated as `stream`'s own (None: the current
    one's); while that stream is being captured, out of the graph's pool."""
    with torch.cuda.device(index), torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device="cuda")


def _on(stream, f, *args):
    """f(*args), its results allocated as `stream`'s own: memory of the current
    stream may still be in use there by work that `stream` does not wait for."""
    with torch.cuda.stream(stream):
        return f(*args)


class CachePlan(NamedTuple):
    """What swiglu_cache_plan makes; pass it as `out` to reuse its buffers, in
    turn with another where pages_held and counts[2:3] go into the next step."""
    query_start: torch.Tensor          # [R + 1] int32
    slots: torch.Tensor                # [max_tokens] int32
    positions: torch.Tensor            # [max_tokens] int32
    pages_held: torch.Tensor           # [R] int32
    counts: torch.Tensor               # [3] int32: tokens, pages wanted, next free_head
    mask: Optional[torch.Tensor]       # [max_tokens, words] int64, or None


def swiglu_cache_plan(ctx_lens: torch.Tensor, new_lens: torch.Tensor, pages_held: torch.Tensor,
                      block_table: torch.Tensor, free_pages: torch.Tensor, page_size: int,
                      max_tokens: int, parents: torch.Tensor = None,
                      free_head: torch.Tensor = None, out: CachePlan = None,
                      stream=None) -> CachePlan:
    """Block tables (in place), slots, positions and tree masks of one step
    from the requests' lengths, in one launch; nothing is read on the host.
    `max_tokens` rows of slots, positions and masks are made (rows past the
    step's tokens: slot -1, mask 0). `free_head` [1] (None: 0) is where the
    free list starts; the next step's is counts[2:3].

    No input may share memory with `out` (SwigluError): every block reads all
    lengths while others write. So a step that takes the last plan's pages_held or
    counts[2:3] fills another plan, and two of them alternate."""
    native = _binding or _native()
    if out is None and stream is not None:
        return _on(stream, swiglu_cache_plan, ctx_lens, new_lens, pages_held, block_table,
                   free_pages, page_size, max_tokens, parents, free_head)
    if out is None:
        if not isinstance(ctx_lens, torch.Tensor):
            raise TypeError("ctx_lens must be a CUDA tensor")
        new, R, T = ctx_lens.new_empty, ctx_lens.numel(), int(max_tokens)
        mask = None if parents is None else new((T, (parents.shape[-1] + 63) // 64),
                                                dtype=torch.int64)
        out = CachePlan(new((R + 1,)), new((T,)), new((T,)), new((R,)), new((3,)), mask)
    native.plan(ctx_lens, new_lens, pages_held, block_table, free_pages, page_size, max_tokens,
                parents, free_head, *out, stream)
    return out


def swiglu_cache_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                       k_cache: torch.Tensor, v_cache: torch.Tensor, stream=None) -> None:
    """Rows of k and v [tokens, kv heads, head size] (strided views allowed)
    into the caches, row t at slots[t]; rows with a negative slot are dropped."""
    (_binding or _native()).write(k, v, slots, k_cache, v_cache, stream)


def swiglu_tree_attention_workspace_bytes(tokens: int, q_heads: int, kv_heads: int,
                                          head_dim: int) -> int:
    return int(load_library().swiglu_tree_attention_workspace_bytes(
        int(tokens), int(q_heads), int(kv_heads), int(head_dim)))


def swiglu_tree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                          block_table: torch.Tensor, ctx_lens: torch.Tensor,
                          query_start: torch.Tensor, mask: torch.Tensor = None,
                          scale: float = None, out: torch.Tensor = None,
                          workspace: torch.Tensor = None, stream=None) -> torch.Tensor:
    """Attention of the step's tokens q [tokens, q heads, head size] over the
    cache, [tokens, q heads, head size] BF16: every token sees its request's
    context and the new tokens in its row of `mask` [tokens, words] int64
    (None: those before it, and itself). The step's own keys and values are
    in the cache already (swiglu_cache_write). `scale` None: 1/sqrt(head size)."""
    attend = (_binding or _native()).attend
    if out is None and stream is not None:
        return _on(stream, attend, q, k_cache, v_cache, block_table, ctx_lens, query_start, mask,
                   scale, out, workspace, None)
    return attend(q, k_cache, v_cache, block_table, ctx_lens, query_start, mask, scale, out,
                  workspace, stream)


def swiglu_cache_accept(k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                        ctx_lens: torch.Tensor, paths: torch.Tensor, path_lens: torch.Tensor,
                        stream=None) -> torch.Tensor:
    """Moves the accepted path's rows (paths [R, width]: increasing indices
    among the request's new tokens, path_lens [R] of them) behind the context,
    in the caches of one layer or of all ([layers, ...]); returns the new
    context lengths."""
    accept = (_binding or _native()).accept
    if stream is not None:
        return _on(stream, accept, k_cache, v_cache, block_table, ctx_lens, paths, path_lens, None)
    return accept(k_cache, v_cache, block_table, ctx_lens, paths, path_lens, None)
