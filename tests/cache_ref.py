"""Plain 64-bit reference of the paged-cache operators (numpy), and builders of
small cases: test infrastructure only."""
from __future__ import annotations

import numpy as np

BF16_U = 2.0 ** -8      # half a unit in the last place of BF16, relative


def bits_to_f64(b):
    return (np.ascontiguousarray(b, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(
        np.float64)


def f32_to_bits(x):
    import workloads
    return workloads.f32_to_bf16_bits(np.asarray(x, np.float32))


def ancestors(parents, n):
    """Bool [n, n]: token i is, or descends from, token j."""
    seen = np.zeros((n, n), bool)
    for i in range(n):
        j = i
        while True:
            seen[i, j] = True
            up = int(parents[j])
            if not 0 <= up < j:
                break
            j = up
    return seen


def pack_words(seen, words):
    """Bool [n, m] -> int64 [n, words], bit j of word j // 64."""
    n, m = seen.shape
    out = np.zeros((n, words), np.uint64)
    for j in range(min(m, 64 * words)):
        out[:, j // 64] |= seen[:, j].astype(np.uint64) << np.uint64(j % 64)
    return out.view(np.int64)


def plan(ctx, new, held, table, free, P, max_tokens, parents=None, head=0):
    """swiglu_cache_plan by its definition; changes `table`."""
    R, max_pages = table.shape
    width = None if parents is None else parents.shape[1]
    words = 0 if parents is None else (width + 63) // 64
    slots = np.full(max_tokens, -1, np.int64)
    positions = np.zeros(max_tokens, np.int64)
    mask = np.zeros((max_tokens, words), np.int64)
    start, held_out, wanted = [0], [], 0
    for r in range(R):
        c, n = max(int(ctx[r]), 0), max(int(new[r]), 0)
        if parents is not None:
            n = min(n, width)
        h = min(max(int(held[r]), 0), max_pages)
        need = max(h, min(max_pages, -(-(c + n) // P)))
        got = 0
        for i in range(need - h):
            at = head + wanted + i
            ok = at < len(free)
            table[r, h + i] = free[at] if ok else -1
            got += ok
        wanted += need - h
        held_out.append(h + got)
        seen = None if parents is None else ancestors(parents[r], n)
        for i in range(n):
            t = start[-1] + i
            if t >= max_tokens:
                continue
            x = c + i
            if x // P < need and table[r, x // P] >= 0:
                slots[t] = int(table[r, x // P]) * P + x % P
            positions[t] = x if seen is None else c + int(seen[i].sum()) - 1
            if seen is not None:
                mask[t] = pack_words(seen[i:i + 1], words)[0]
        start.append(start[-1] + n)
    counts = [start[-1], wanted, head + min(wanted, max(len(free) - head, 0))]
    return {"query_start": np.array(start), "slots": slots, "positions": positions,
            "pages_held": np.array(held_out, np.int64), "counts": np.array(counts),
            "mask": mask, "table": table}


def gather(cache, table_row, L, P, head):
    """Positions 0 .. L - 1 of one head, [L, D], from a cache [pages, heads, P, D]."""
    x = np.arange(L)
    return cache[table_row[x // P], head, x % P]


def attend(q, k, v, table, ctx, start, visible, scale, P):
    """(out, bound) in float64. q [T, Hq, D], k and v [pages, Hkv, P, D];
    visible[r]: bool [n, n] of the new tokens. Positions that a row does not
    see take no part. bound: how far a BF16 result with BF16-rounded weights
    may be: the weights' rounding moves a sum by at most BF16_U * sum p|v| / sum
    p, the final rounding by BF16_U * |o|; 1/8 more for the FP32 steps (scores,
    exponentials and sums, each below 2^-14 relative here) and their products."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, bound = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    for r in range(len(ctx)):
        t0, t1 = int(start[r]), int(start[r + 1])
        n, c = t1 - t0, max(int(ctx[r]), 0)
        L = min(c + n, table.shape[1] * P)
        for h in range(k.shape[1]):
            kk, vv = gather(k, table[r], L, P, h), gather(v, table[r], L, P, h)
            for i in range(n):
                seen = np.ones(L, bool)
                seen[c:] = visible[r][i][: max(L - c, 0)]
                if not seen.any():
                    continue
                for g in range(G):
                    with np.errstate(all="ignore"):
                        s = scale * (kk[seen] @ q[t0 + i, h * G + g])
                        m = s.max()
                        if m == -np.inf:
                            continue
                        p = np.exp(s - m)
                        o = (p @ vv[seen]) / p.sum()
                        b = (p @ np.abs(vv[seen])) / p.sum()
                    out[t0 + i, h * G + g] = o
                    bound[t0 + i, h * G + g] = 1.125 * BF16_U * (b + np.abs(o)) + 1e-30
    return out, bound


def accept(caches, table, ctx, paths, lens, P):
    """New copies of caches [layers, pages, heads, P, D] after the move."""
    done = []
    for cache in caches:
        new = cache.copy()
        for r in range(len(ctx)):
            for i in range(min(max(int(lens[r]), 0), paths.shape[1])):
                a, b = int(ctx[r]) + int(paths[r, i]), int(ctx[r]) + i
                new[:, table[r, b // P], :, b % P] = cache[:, table[r, a // P], :, a % P]
        done.append(new)
    return done


def tables(rng, need, pages, extra=1):
    """Random distinct pages for each request: [R, max(need) + extra], -1 past."""
    perm = rng.permutation(pages)
    table = np.full((len(need), int(max(need, default=0)) + extra), -1, np.int32)
    at = 0
    for r, m in enumerate(need):
        table[r, :m] = perm[at:at + m]
        at += m
    return table


def random_parents(rng, n):
    par = np.full(n, -1, np.int32)
    for i in range(1, n):
        par[i] = rng.integers(-1, i)
    return par
