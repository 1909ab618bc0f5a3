"""Binding of the paged-cache entry points: argument checks and marshalling
only, as in the package's __init__ (include/swiglu.h has the contracts).

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

from typing import NamedTuple, Optional

import torch

from . import (SWIGLU_ERR_INVALID_ARG, SwigluError, _check, _OnDevice, _out_tensor,
               _require_bf16_cuda, _stream_handle, load_library)

# (device index, stream handle) -> uint8 tensor; apart from the other entry
# points' workspaces, whose counters have to stay as they are between calls
_workspaces = {}


class CachePlan(NamedTuple):
    """What swiglu_cache_plan makes; pass it as `out` to reuse its buffers."""
    query_start: torch.Tensor          # [R + 1] int32
    slots: torch.Tensor                # [max_tokens] int32
    positions: torch.Tensor            # [max_tokens] int32
    pages_held: torch.Tensor           # [R] int32
    counts: torch.Tensor               # [3] int32: tokens, pages wanted, next free_head
    mask: Optional[torch.Tensor]       # [max_tokens, words] int64, or None


def _require_ints(t, name: str, device, shape, dtype=torch.int32):
    """An int32 (or `dtype`) CUDA tensor on `device`, contiguous, of `shape`
    (None: any extent)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s must be on %s" % (name, device))
    got = t.shape
    if len(got) != len(shape) or any(b is not None and a != b for a, b in zip(got, shape)):
        raise ValueError("%s must be %s, got %s" % (
            name, [("any" if b is None else b) for b in shape], list(got)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _require_rows(t, name: str, device, heads=None, dim=None):
    """A [tokens, heads, head size] BF16 view: any strides of the first two
    dimensions that are multiples of 8, the last one contiguous."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype is not torch.bfloat16:
        raise TypeError("%s must be bfloat16, got %s" % (name, t.dtype))
    if t.device != device:
        raise ValueError("%s must be on %s" % (name, device))
    shape = t.shape
    if len(shape) != 3 or (heads is not None and shape[1] != heads) or (
            dim is not None and shape[2] != dim):
        raise ValueError("%s must be [tokens, %s, %s], got %s" % (
            name, "heads" if heads is None else heads, "head size" if dim is None else dim,
            list(shape)))
    s = t.stride()
    if s[2] != 1 or s[0] % 8 or s[1] % 8:
        raise ValueError("%s must have a contiguous last dimension and strides that are "
                         "multiples of 8, got strides %s" % (name, s))
    return s


def _require_caches(k_cache, v_cache, layered: bool):
    _require_bf16_cuda(k_cache, "k_cache")
    _require_bf16_cuda(v_cache, "v_cache")
    dims = k_cache.dim()
    if (dims != 4 and not (layered and dims == 5)) or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must both be [%spages, kv heads, page size, "
                         "head size]" % ("layers, " if layered and dims == 5 else ""))
    if v_cache.device != k_cache.device:
        raise ValueError("v_cache must be on %s" % k_cache.device)
    return k_cache.shape


def swiglu_cache_plan(ctx_lens: torch.Tensor, new_lens: torch.Tensor, pages_held: torch.Tensor,
                      block_table: torch.Tensor, free_pages: torch.Tensor, page_size: int,
                      max_tokens: int, parents: torch.Tensor = None,
                      free_head: torch.Tensor = None, out: CachePlan = None,
                      stream=None) -> CachePlan:
    """Block tables (in place), slots, positions and tree masks of one step
    from the requests' lengths, in one launch; nothing is read on the host.
    `max_tokens` rows of slots, positions and masks are made (rows past the
    step's tokens: slot -1, mask 0). `free_head` [1] (None: 0) is where the
    free list starts; the next step's is counts[2:3]."""
    lib = load_library()
    dev = ctx_lens.device if isinstance(ctx_lens, torch.Tensor) else None
    _require_ints(ctx_lens, "ctx_lens", dev, (None,))
    R = ctx_lens.shape[0]
    max_tokens = int(max_tokens)
    _require_ints(new_lens, "new_lens", dev, (R,))
    _require_ints(pages_held, "pages_held", dev, (R,))
    _require_ints(block_table, "block_table", dev, (R, None))
    _require_ints(free_pages, "free_pages", dev, (None,))
    if free_head is not None:
        _require_ints(free_head, "free_head", dev, (1,))
    width = words = 0
    if parents is not None:
        _require_ints(parents, "parents", dev, (R, None))
        width = parents.shape[1]
        words = (width + 63) // 64
        if width == 0:
            raise ValueError("parents must have at least one column")
    if out is None:
        i32 = {"dtype": torch.int32, "device": dev}
        out = CachePlan(torch.empty(R + 1, **i32), torch.empty(max_tokens, **i32),
                        torch.empty(max_tokens, **i32), torch.empty(R, **i32),
                        torch.empty(3, **i32),
                        None if parents is None else torch.empty(
                            (max_tokens, words), dtype=torch.int64, device=dev))
    else:
        _require_ints(out.query_start, "out.query_start", dev, (R + 1,))
        _require_ints(out.slots, "out.slots", dev, (max_tokens,))
        _require_ints(out.positions, "out.positions", dev, (max_tokens,))
        _require_ints(out.pages_held, "out.pages_held", dev, (R,))
        _require_ints(out.counts, "out.counts", dev, (3,))
        if (out.mask is None) != (parents is None):
            raise ValueError("out.mask goes with parents: both or neither")
        if parents is not None:
            _require_ints(out.mask, "out.mask", dev, (max_tokens, words), torch.int64)
    with _OnDevice(dev):
        _check(lib.swiglu_cache_plan(
            ctx_lens.data_ptr(), new_lens.data_ptr(), pages_held.data_ptr(),
            block_table.data_ptr(), R, block_table.shape[1], free_pages.data_ptr(),
            free_pages.shape[0], None if free_head is None else free_head.data_ptr(),
            int(page_size), None if parents is None else parents.data_ptr(), width, max_tokens,
            out.query_start.data_ptr(), out.slots.data_ptr(), out.positions.data_ptr(),
            out.pages_held.data_ptr(), out.counts.data_ptr(),
            None if parents is None else out.mask.data_ptr(), _stream_handle(stream)),
            "swiglu_cache_plan")
    return out


def swiglu_cache_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                       k_cache: torch.Tensor, v_cache: torch.Tensor, stream=None) -> None:
    """Rows of k and v [tokens, kv heads, head size] (strided views allowed)
    into the caches, row t at slots[t]; rows with a negative slot are dropped."""
    lib = load_library()
    pages, heads, page_size, dim = _require_caches(k_cache, v_cache, False)
    dev = k_cache.device
    ks = _require_rows(k, "k", dev, heads, dim)
    vs = _require_rows(v, "v", dev, heads, dim)
    T = k.shape[0]
    if v.shape[0] != T:
        raise ValueError("k and v must have the same number of tokens")
    _require_ints(slots, "slots", dev, (T,))
    with _OnDevice(dev):
        _check(lib.swiglu_cache_write(
            k.data_ptr(), v.data_ptr(), T, heads, dim, ks[0], ks[1], vs[0], vs[1],
            slots.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), pages, page_size,
            _stream_handle(stream)), "swiglu_cache_write")


def swiglu_tree_attention_workspace_bytes(tokens: int, q_heads: int, kv_heads: int,
                                          head_dim: int) -> int:
    return int(load_library().swiglu_tree_attention_workspace_bytes(
        int(tokens), int(q_heads), int(kv_heads), int(head_dim)))


def _workspace(device, nbytes: int, stream) -> torch.Tensor:
    """One attention workspace per (device, stream), grown on demand."""
    s = torch.cuda.current_stream(device) if stream is None else stream
    key = (device.index, int(s.cuda_stream))
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        if torch.cuda.is_current_stream_capturing():
            # an allocation made during capture belongs to the graph's pool
            raise SwigluError(SWIGLU_ERR_INVALID_ARG,
                              "this call needs a workspace of %d bytes: allocate it before "
                              "capturing (swiglu_tree_attention_workspace_bytes) and pass "
                              "workspace=" % nbytes)
        with torch.cuda.stream(s):
            ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


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
    lib = load_library()
    pages, kv_heads, page_size, dim = _require_caches(k_cache, v_cache, False)
    dev = k_cache.device
    qs = _require_rows(q, "q", dev, None, dim)
    T, heads = q.shape[0], q.shape[1]
    if heads % kv_heads:
        raise ValueError("q heads (%d) must be a multiple of kv heads (%d)" % (heads, kv_heads))
    _require_ints(ctx_lens, "ctx_lens", dev, (None,))
    R = ctx_lens.shape[0]
    _require_ints(block_table, "block_table", dev, (R, None))
    _require_ints(query_start, "query_start", dev, (R + 1,))
    words = 0
    if mask is not None:
        _require_ints(mask, "mask", dev, (T, None), torch.int64)
        words = mask.shape[1]
        if words == 0:
            raise ValueError("mask must have at least one word a token")
    out = _out_tensor(out, (T, heads, dim), dev, "out")
    with _OnDevice(dev):
        need = lib.swiglu_tree_attention_workspace_bytes(T, heads, kv_heads, dim)
        ws_ptr, ws_bytes = None, 0
        if need:
            if workspace is None:
                workspace = _workspace(dev, need, stream)
            ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        _check(lib.swiglu_tree_attention(
            q.data_ptr(), qs[0], qs[1], k_cache.data_ptr(), v_cache.data_ptr(), pages, page_size,
            block_table.data_ptr(), R, block_table.shape[1], ctx_lens.data_ptr(),
            query_start.data_ptr(), None if mask is None else mask.data_ptr(), words,
            dim ** -0.5 if scale is None else float(scale), out.data_ptr(), T, heads, kv_heads,
            dim, ws_ptr, ws_bytes, _stream_handle(stream)), "swiglu_tree_attention")
    return out


def swiglu_cache_accept(k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                        ctx_lens: torch.Tensor, paths: torch.Tensor, path_lens: torch.Tensor,
                        stream=None) -> torch.Tensor:
    """Moves the accepted path's rows (paths [R, width]: increasing indices
    among the request's new tokens, path_lens [R] of them) behind the context,
    in the caches of one layer or of all ([layers, ...]); returns the new
    context lengths."""
    lib = load_library()
    shape = _require_caches(k_cache, v_cache, True)
    layers = shape[0] if len(shape) == 5 else 1
    pages, heads, page_size, dim = shape[-4:]
    dev = k_cache.device
    _require_ints(ctx_lens, "ctx_lens", dev, (None,))
    R = ctx_lens.shape[0]
    _require_ints(block_table, "block_table", dev, (R, None))
    _require_ints(paths, "paths", dev, (R, None))
    _require_ints(path_lens, "path_lens", dev, (R,))
    new_ctx = torch.empty_like(ctx_lens)
    with _OnDevice(dev):
        _check(lib.swiglu_cache_accept(
            k_cache.data_ptr(), v_cache.data_ptr(), layers, pages, heads, page_size, dim,
            block_table.data_ptr(), R, block_table.shape[1], ctx_lens.data_ptr(),
            paths.data_ptr(), paths.shape[1], path_lens.data_ptr(), new_ctx.data_ptr(),
            _stream_handle(stream)), "swiglu_cache_accept")
    return new_ctx
