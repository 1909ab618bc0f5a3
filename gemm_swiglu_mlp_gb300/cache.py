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

from . import SWIGLU_ERR_INVALID_ARG, SWIGLU_OK, SwigluError, load_library

# These calls are a few microseconds of GPU time in a serving step, so the
# binding keeps its own small: one comparison per tensor on the way that
# succeeds (what is wrong is worked out only for the message), and the current
# stream's handle without a Stream object (~3 us).
_I32, _I64, _BF16 = torch.int32, torch.int64, torch.bfloat16
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)

# (device index, stream handle) -> uint8 tensor; apart from the other entry
# points' workspaces, whose counters have to stay as they are between calls
_workspaces = {}
_ws_bytes = {}     # (device index, tokens, q heads, kv heads, head size) -> bytes


class CachePlan(NamedTuple):
    """What swiglu_cache_plan makes; pass it as `out` to reuse its buffers."""
    query_start: torch.Tensor          # [R + 1] int32
    slots: torch.Tensor                # [max_tokens] int32
    positions: torch.Tensor            # [max_tokens] int32
    pages_held: torch.Tensor           # [R] int32
    counts: torch.Tensor               # [3] int32: tokens, pages wanted, next free_head
    mask: Optional[torch.Tensor]       # [max_tokens, words] int64, or None


def _refuse(t, name: str, index: int, dtype, shape, contiguous=True):
    """Says what is wrong with a tensor that one of the checks below refused."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.get_device() != index:
        raise ValueError("%s must be on cuda:%d, got %s" % (name, index, t.device))
    if contiguous and not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    raise ValueError("%s must be %s, got %s" % (name, shape, list(t.shape)))


def _vector(t, name: str, n, index: int):
    """A contiguous int32 CUDA vector of n values (None: any) on device
    `index` (-1: any); returns its length and device."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is _I32 and t.is_contiguous():
        shape, at = t.shape, t.get_device()
        if len(shape) == 1 and (n is None or shape[0] == n) and (index < 0 or at == index):
            return shape[0], at
    _refuse(t, name, index if index >= 0 else 0, _I32, "[%s]" % ("any" if n is None else n))


def _matrix(t, name: str, rows: int, index: int, dtype=_I32) -> int:
    """A contiguous CUDA matrix of `rows` rows; returns its columns (>= 1)."""
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.is_contiguous()
            and t.get_device() == index):
        shape = t.shape
        if len(shape) == 2 and shape[0] == rows and shape[1] > 0:
            return shape[1]
    _refuse(t, name, index, dtype, "[%d, at least 1]" % rows)


def _rows(t, name: str, index: int, tokens, heads, dim: int):
    """A [tokens, heads, dim] BF16 view (None: any) whose last dimension is
    contiguous, any strides of the others that are multiples of 8; returns
    (shape, strides)."""
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is _BF16
            and t.get_device() == index):
        shape = t.shape
        if (len(shape) == 3 and shape[2] == dim and (heads is None or shape[1] == heads)
                and (tokens is None or shape[0] == tokens)):
            s = t.stride()
            if s[2] == 1 and not (s[0] | s[1]) & 7:
                return shape, s
            raise ValueError("%s must have a contiguous last dimension and strides that are "
                             "multiples of 8, got strides %s" % (name, s))
    _refuse(t, name, index, _BF16, "[%s, %s, %d]" % (
        "tokens" if tokens is None else tokens, "heads" if heads is None else heads, dim), False)


def _caches(k_cache, v_cache, layered: bool):
    """(shape, device index) of a pair of caches."""
    if (isinstance(k_cache, torch.Tensor) and k_cache.is_cuda and k_cache.dtype is _BF16
            and k_cache.is_contiguous()):
        shape, index = k_cache.shape, k_cache.get_device()
        if len(shape) == 4 or (layered and len(shape) == 5):
            if (isinstance(v_cache, torch.Tensor) and v_cache.is_cuda and v_cache.dtype is _BF16
                    and v_cache.is_contiguous() and v_cache.shape == shape
                    and v_cache.get_device() == index):
                return shape, index
            _refuse(v_cache, "v_cache", index, _BF16, list(shape))
    _refuse(k_cache, "k_cache", k_cache.get_device() if isinstance(k_cache, torch.Tensor) else 0,
            _BF16, "[%spages, kv heads, page size, head size]" % ("layers, " if layered else ""))


def _call(entry: str, fn, index: int, stream, *args):
    """fn(*args, stream handle) with device `index` current."""
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return _call(entry, fn, index, stream, *args)
    status = fn(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    if status != SWIGLU_OK:
        raise SwigluError(status, entry)


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
    R, index = _vector(ctx_lens, "ctx_lens", None, -1)
    T = int(max_tokens)
    _vector(new_lens, "new_lens", R, index)
    _vector(pages_held, "pages_held", R, index)
    if R or block_table.dim() != 2:
        max_pages = _matrix(block_table, "block_table", R, index)
    else:
        max_pages = max(block_table.shape[1], 1)
    num_free, _ = _vector(free_pages, "free_pages", None, index)
    head_ptr = par_ptr = mask_ptr = None
    if free_head is not None:
        _vector(free_head, "free_head", 1, index)
        head_ptr = free_head.data_ptr()
    width = words = 0
    if parents is not None:
        width = _matrix(parents, "parents", R, index)
        words = (width + 63) // 64
        par_ptr = parents.data_ptr()
    if out is None:
        new = ctx_lens.new_empty
        out = CachePlan(new((R + 1,)), new((T,)), new((T,)), new((R,)), new((3,)),
                        None if parents is None else new((T, words), dtype=_I64))
    else:
        _vector(out.query_start, "out.query_start", R + 1, index)
        _vector(out.slots, "out.slots", T, index)
        _vector(out.positions, "out.positions", T, index)
        _vector(out.pages_held, "out.pages_held", R, index)
        _vector(out.counts, "out.counts", 3, index)
        if (out.mask is None) != (parents is None):
            raise ValueError("out.mask goes with parents: both or neither")
    if parents is not None:
        if T and _matrix(out.mask, "out.mask", T, index, _I64) != words:
            raise ValueError("out.mask must be [%d, %d]" % (T, words))
        mask_ptr = out.mask.data_ptr()
    _call("swiglu_cache_plan", load_library().swiglu_cache_plan, index, stream,
          ctx_lens.data_ptr(), new_lens.data_ptr(), pages_held.data_ptr(), block_table.data_ptr(),
          R, max_pages, free_pages.data_ptr(), num_free, head_ptr, int(page_size), par_ptr, width,
          T, out.query_start.data_ptr(), out.slots.data_ptr(), out.positions.data_ptr(),
          out.pages_held.data_ptr(), out.counts.data_ptr(), mask_ptr)
    return out


def swiglu_cache_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                       k_cache: torch.Tensor, v_cache: torch.Tensor, stream=None) -> None:
    """Rows of k and v [tokens, kv heads, head size] (strided views allowed)
    into the caches, row t at slots[t]; rows with a negative slot are dropped."""
    (pages, heads, page_size, dim), index = _caches(k_cache, v_cache, False)
    shape, ks = _rows(k, "k", index, None, heads, dim)
    T = shape[0]
    _, vs = _rows(v, "v", index, T, heads, dim)
    _vector(slots, "slots", T, index)
    _call("swiglu_cache_write", load_library().swiglu_cache_write, index, stream,
          k.data_ptr(), v.data_ptr(), T, heads, dim, ks[0], ks[1], vs[0], vs[1], slots.data_ptr(),
          k_cache.data_ptr(), v_cache.data_ptr(), pages, page_size)


def swiglu_tree_attention_workspace_bytes(tokens: int, q_heads: int, kv_heads: int,
                                          head_dim: int) -> int:
    return int(load_library().swiglu_tree_attention_workspace_bytes(
        int(tokens), int(q_heads), int(kv_heads), int(head_dim)))


def _workspace(index: int, nbytes: int, stream) -> torch.Tensor:
    """One attention workspace per (device, stream), grown on demand."""
    handle = _raw_stream(index) if stream is None else stream.cuda_stream
    ws = _workspaces.get((index, handle))
    if ws is None or ws.numel() < nbytes:
        if torch.cuda.is_current_stream_capturing():
            # an allocation made during capture belongs to the graph's pool
            raise SwigluError(SWIGLU_ERR_INVALID_ARG,
                              "this call needs a workspace of %d bytes: allocate it before "
                              "capturing (swiglu_tree_attention_workspace_bytes) and pass "
                              "workspace=" % nbytes)
        with torch.cuda.device(index), torch.cuda.stream(stream):
            ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        _workspaces[index, handle] = ws
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
    (pages, kv_heads, page_size, dim), index = _caches(k_cache, v_cache, False)
    shape, qs = _rows(q, "q", index, None, None, dim)
    T, heads, _ = shape
    if heads % kv_heads:
        raise ValueError("q heads (%d) must be a multiple of kv heads (%d)" % (heads, kv_heads))
    R, _ = _vector(ctx_lens, "ctx_lens", None, index)
    if R or block_table.dim() != 2:
        max_pages = _matrix(block_table, "block_table", R, index)
    else:
        max_pages = max(block_table.shape[1], 1)
    _vector(query_start, "query_start", R + 1, index)
    words, mask_ptr = 0, None
    if mask is not None:
        words = _matrix(mask, "mask", T, index, _I64)
        mask_ptr = mask.data_ptr()
    if out is None:
        out = torch.empty(shape, dtype=_BF16, device=q.device)
    elif (not isinstance(out, torch.Tensor) or not out.is_cuda or out.dtype is not _BF16
          or out.shape != shape or not out.is_contiguous() or out.get_device() != index):
        _refuse(out, "out", index, _BF16, list(shape))
    key = (index, T, heads, kv_heads, dim)
    need = _ws_bytes.get(key)
    if need is None:
        with torch.cuda.device(index):
            need = _ws_bytes[key] = swiglu_tree_attention_workspace_bytes(T, heads, kv_heads, dim)
    ws_ptr, ws_bytes = None, 0
    if need:
        if workspace is None:
            workspace = _workspace(index, need, stream)
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _call("swiglu_tree_attention", load_library().swiglu_tree_attention, index, stream,
          q.data_ptr(), qs[0], qs[1], k_cache.data_ptr(), v_cache.data_ptr(), pages, page_size,
          block_table.data_ptr(), R, max_pages, ctx_lens.data_ptr(), query_start.data_ptr(),
          mask_ptr, words, dim ** -0.5 if scale is None else float(scale), out.data_ptr(), T,
          heads, kv_heads, dim, ws_ptr, ws_bytes)
    return out


def swiglu_cache_accept(k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                        ctx_lens: torch.Tensor, paths: torch.Tensor, path_lens: torch.Tensor,
                        stream=None) -> torch.Tensor:
    """Moves the accepted path's rows (paths [R, width]: increasing indices
    among the request's new tokens, path_lens [R] of them) behind the context,
    in the caches of one layer or of all ([layers, ...]); returns the new
    context lengths."""
    shape, index = _caches(k_cache, v_cache, True)
    layers = shape[0] if len(shape) == 5 else 1
    pages, heads, page_size, dim = shape[-4:]
    R, _ = _vector(ctx_lens, "ctx_lens", None, index)
    max_pages = _matrix(block_table, "block_table", R, index)
    width = _matrix(paths, "paths", R, index)
    _vector(path_lens, "path_lens", R, index)
    new_ctx = torch.empty_like(ctx_lens)
    _call("swiglu_cache_accept", load_library().swiglu_cache_accept, index, stream,
          k_cache.data_ptr(), v_cache.data_ptr(), layers, pages, heads, page_size, dim,
          block_table.data_ptr(), R, max_pages, ctx_lens.data_ptr(), paths.data_ptr(), width,
          path_lens.data_ptr(), new_ctx.data_ptr())
    return new_ctx
