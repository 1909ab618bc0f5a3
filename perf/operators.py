"""Cases of the drafted-token serving operators: what is measured and checked.

Four operators serve one verification step of a batch of requests whose keys
and values lie in a paged cache:

  plan    block tables, slot map, positions and tree masks from the requests'
          lengths and their draft trees (whole numbers)
  write   the step's new keys and values into the cache, by the slot map
  attend  attention of the step's tokens over the cache: every token sees its
          request's context and, of the step's own tokens, its ancestors in
          the tree (or, without a tree, the tokens before it) and itself
  accept  the accepted path's keys and values moved to the rows right after
          the context, in every layer at once

Cache layout: K and V each [pages, kv heads, page size, head size], BF16.
``run`` computes a case in plain torch operations (``own`` false) or through
the package's entry points (``own`` true).
"""
import math

import numpy as np
import torch

own = False
DEV = "cuda"


# ----------------------------------------------------------------- cases
def listed():
    return [
        # one user's next token, a small model (896 = 14 heads of 64): launch and latency
        {"name": "attend_one", "op": "attend", "R": 1, "n": 1, "lo": 700, "hi": 700, "hq": 14,
         "hkv": 2, "D": 64, "P": 16, "tree": False, "lens": 1},
        # ordinary decoding of a batch (3584 = 28 heads of 128), ragged contexts
        {"name": "attend_decode", "op": "attend", "R": 64, "n": 1, "lo": 500, "hi": 8000, "hq": 28,
         "hkv": 4, "D": 128, "P": 16, "tree": False, "lens": 2},
        # a few users' small trees (1536 = 12 heads of 128)
        {"name": "attend_tree_few", "op": "attend", "R": 4, "n": 13, "lo": 300, "hi": 3000,
         "hq": 12, "hkv": 2, "D": 128, "P": 32, "tree": True, "lens": 3},
        # a full batch of large trees (8192 = 64 heads of 128): arithmetic counts
        {"name": "attend_tree_large", "op": "attend", "R": 32, "n": 64, "lo": 2000, "hi": 6000,
         "hq": 64, "hkv": 8, "D": 128, "P": 64, "tree": True, "lens": 4},
        # two very long documents with a tree each (5120 = 40 heads of 128): one stream of K and V
        {"name": "attend_long", "op": "attend", "R": 2, "n": 25, "lo": 131072, "hi": 131072,
         "hq": 40, "hkv": 8, "D": 128, "P": 64, "tree": True, "lens": 5},
        # pieces of prompts (causal chains), some of them the prompt's beginning
        {"name": "attend_chain", "op": "attend", "R": 6, "n": 200, "lo": 1, "hi": 2000, "hq": 28,
         "hkv": 4, "D": 128, "P": 16, "tree": False, "lens": 6},
        # bookkeeping of a decoding batch, one token a request
        {"name": "plan_decode", "op": "plan", "R": 64, "n": 1, "lo": 500, "hi": 8000, "P": 16,
         "tree": False, "lens": 2},
        # bookkeeping of a large batch of trees
        {"name": "plan_tree", "op": "plan", "R": 192, "n": 60, "lo": 100, "hi": 8000, "P": 16,
         "tree": True, "lens": 7},
        # the new rows of a batch of trees
        {"name": "write_tree", "op": "write", "R": 48, "n": 45, "lo": 100, "hi": 500, "hkv": 4,
         "D": 128, "P": 16, "tree": True, "lens": 8},
        # the new rows of whole prompts
        {"name": "write_prompt", "op": "write", "R": 10, "n": 2000, "lo": 1, "hi": 50, "hkv": 8,
         "D": 128, "P": 64, "tree": False, "lens": 9},
        # the accepted paths of a few requests, one layer
        {"name": "accept_few", "op": "accept", "R": 8, "n": 13, "lo": 100, "hi": 1000, "hkv": 2,
         "D": 128, "P": 32, "layers": 1, "tree": True, "lens": 10},
        # the accepted paths of a batch, every layer of a model
        {"name": "accept_layers", "op": "accept", "R": 48, "n": 45, "lo": 100, "hi": 500, "hkv": 4,
         "D": 128, "P": 16, "layers": 28, "tree": True, "lens": 11},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "attend", "plan", "write", "accept"])
    c = {"op": op, "R": _log(rng, 1, 200), "P": rng.choice([16, 32, 64, 128]),
         "tree": rng.random() < 0.6 or op == "accept", "lens": rng.randrange(1 << 20)}
    c["n"] = _log(rng, 2, 64) if c["tree"] else (1 if rng.random() < 0.5 else _log(rng, 2, 300))
    if op == "attend" and rng.random() < 0.25:
        c["R"] = rng.randint(1, 4)
    c["hi"] = _log(rng, 50, 130000 if c["R"] <= 4 and op == "attend" else 8000)
    c["lo"] = _log(rng, 1, c["hi"])
    if op == "plan":
        return c
    c["hkv"] = rng.choice([1, 2, 4, 8])
    c["D"] = rng.choice([64, 128])
    if op == "attend":
        c["hq"] = c["hkv"] * rng.choice([1, 2, 4, 5, 6, 7, 8])
        # no more keys and values or products than the largest listed cases
        while (4 * c["R"] * (c["hi"] + c["n"]) * c["hkv"] * c["D"] > 1.0e9
               or 4 * c["R"] * (c["hi"] + c["n"]) * c["n"] * c["hq"] * c["D"] > 2.0e11):
            if c["hi"] > 50:
                c["hi"] = max(50, c["hi"] // 2)
            else:
                c["R"] = max(1, c["R"] // 2)
        c["lo"] = min(c["lo"], c["hi"])
        return c
    c["hi"], c["lo"] = min(c["hi"], 500), min(c["lo"], 500)
    if op == "accept":
        c["R"], c["n"] = min(c["R"], 48), max(c["n"], 4)
        c["layers"] = _log(rng, 1, min(28, 112 // c["hkv"]))
    else:
        c["n"] = max(1, min(c["n"], 20000 // c["R"]))
    return c


# ----------------------------------------------------------------- sizes and inputs
def _lengths(c):
    """Context and new-token counts of each request, from the case alone."""
    r = np.random.RandomState(c["lens"])
    ctx = np.exp(r.uniform(np.log(c["lo"]), np.log(c["hi"] + 1e-9), c["R"])).round().astype(np.int64)
    new = np.full(c["R"], c["n"], np.int64)
    if c["n"] > 1:  # ragged, the first one full
        new = r.randint(max(1, (c["n"] + 1) // 2), c["n"] + 1, c["R"])
        new[0] = c["n"]
    return ctx, new


def _trees(c, new, r):
    """Parents [R, n] (index among the request's new tokens, -1: the context)."""
    par = np.full((c["R"], c["n"]), -1, np.int64)
    i = np.arange(1, c["n"])
    par[:, 1:] = i // 3 + (r.random_sample((c["R"], c["n"] - 1)) * (i - i // 3)).astype(np.int64)
    par[np.arange(c["n"])[None, :] >= new[:, None]] = -1
    return par


def _mask_words(par, new):
    """Ancestor bits (and the token's own) of every new token, [T, words] int64."""
    R, n = par.shape
    anc = np.zeros((R, n, n), bool)
    rows = np.arange(R)
    for i in range(n):
        has = par[:, i] >= 0
        anc[has, i] = anc[rows[has], par[has, i]]
        anc[:, i, i] = True
    W = (n + 63) // 64
    bits = np.zeros((R, n, 64 * W), np.uint64)
    bits[:, :, :n] = anc
    words = (bits.reshape(R, n, W, 64) << np.arange(64, dtype=np.uint64)).sum(-1, dtype=np.uint64)
    keep = np.arange(n)[None, :] < new[:, None]
    return words[keep].view(np.int64)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _tables(c, ctx, new, r):
    """Every request's pages in a random order: [R, max pages] (-1 past the
    pages in use), the number of pages of the cache and the pages used."""
    need = (ctx + new + c["P"] - 1) // c["P"]
    pages = int(need.sum()) + 8
    perm = r.permutation(pages)
    table = np.full((c["R"], int(need.max()) + 1), -1, np.int64)
    held = np.arange(table.shape[1])[None, :] < need[:, None]
    table[held] = perm[: int(need.sum())]
    return table, pages, need


def _normal(g, shape, scale=1.0):
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    return x if scale == 1.0 else x * scale


def prepare(case, seed):
    c = dict(case)
    r = np.random.RandomState(seed % (1 << 32))
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    ctx, new = _lengths(c)
    start = np.concatenate([[0], np.cumsum(new)])
    T = int(start[-1])
    table, pages, need = _tables(c, ctx, new, r)
    s = {"c": c, "T": T, "ctx": _i32(ctx), "new": _i32(new), "start": _i32(start)}
    if c["op"] == "plan":
        held = (ctx + c["P"] - 1) // c["P"]
        lead = np.arange(table.shape[1])[None, :] < held[:, None]
        free = r.permutation(np.concatenate([table[(table >= 0) & ~lead],
                                             pages + np.arange(64)]))
        s["table"] = _i32(np.where(lead, table, -1))
        s["held"], s["free"] = _i32(held), _i32(free)
        s["parents"] = _i32(_trees(c, new, r)) if c["tree"] else None
        s["plan"] = None  # the outputs of the last pass, used again by the next
        return s
    s["table"] = _i32(table)
    shape = (pages, c["hkv"], c["P"], c["D"])
    if c["op"] == "attend":
        s["k"], s["v"] = _normal(g, shape), _normal(g, shape)
        s["q"] = _normal(g, (T, c["hq"], c["D"]), 1.5)
        words = _mask_words(_trees(c, new, r), new) if c["tree"] else None
        s["mask"] = torch.from_numpy(words).to(DEV) if c["tree"] else None
    elif c["op"] == "write":
        s["k"], s["v"] = _normal(g, shape), _normal(g, shape)
        # keys and values as a fused projection leaves them, [T, 2, heads, D]
        s["kv"] = _normal(g, (T, 2, c["hkv"], c["D"]))
        at = np.concatenate([np.arange(a, a + m) for a, m in zip(ctx, new)])
        req = np.repeat(np.arange(c["R"]), new)
        s["slots"] = _i32(table[req, at // c["P"]] * c["P"] + at % c["P"])
    else:
        s["k"], s["v"] = (_normal(g, (c["layers"],) + shape) for _ in range(2))
        # a path keeps its first tokens in place and takes the others from behind the
        # rows that it fills, so that a second pass moves the same values again
        depth = max(2, min(6, c["n"] // 4))
        paths, lens = np.full((c["R"], depth), -1, np.int64), np.zeros(c["R"], np.int64)
        for i in range(c["R"]):
            p = r.randint(1, min(depth, max(1, new[i] // 2)) + 1)
            stay = r.randint(1, p + 1)
            rest = np.sort(r.choice(np.arange(p, new[i]), p - stay, replace=False))
            paths[i, :p] = np.concatenate([np.arange(stay), rest])
            lens[i] = p
        s["paths"], s["lens"] = _i32(paths), _i32(lens)
    return s


# ----------------------------------------------------------------- plain forms
def _request_of(start, T, R):
    t = torch.arange(T, device=DEV)
    return torch.searchsorted(start[1:].long(), t, right=True).clamp(max=R - 1), t


def _plain_plan(s):
    c, T = s["c"], s["T"]
    P, R = c["P"], c["R"]
    ctx, new, held, free = (s[k].long() for k in ("ctx", "new", "held", "free"))
    need = torch.maximum((ctx + new + P - 1) // P, held)
    first = torch.cumsum(need - held, 0) - (need - held)
    start = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.cumsum(new, 0)])
    col = torch.arange(s["table"].shape[1], device=DEV)
    fresh = (col[None, :] >= held[:, None]) & (col[None, :] < need[:, None])
    take = (first[:, None] + col[None, :] - held[:, None]).clamp(0, free.numel() - 1)
    table = torch.where(fresh, free[take].int(), s["table"])
    s["table"].copy_(table)
    req, t = _request_of(start, T, R)
    i = t - start[req]
    at = ctx[req] + i
    slots = (table[req, at // P].long() * P + at % P).int()
    pages = (need - held).sum()
    counts = torch.stack([start[-1], pages, pages]).int()
    out = {"table": s["table"], "start": start.int(), "slots": slots, "held": need.int(),
           "counts": counts}
    if s["parents"] is None:
        out["positions"] = at.int()
        return out
    par, n = s["parents"].long(), c["n"]
    W = (n + 63) // 64
    hop = (par[:, :, None] == torch.arange(n, device=DEV)).float()
    seen = torch.linalg.matrix_power(hop + torch.eye(n, device=DEV), n) > 0
    seen = torch.nn.functional.pad(seen, (0, 64 * W - n)).view(R, n, W, 64)
    words = (seen.long() << torch.arange(64, device=DEV)).sum(-1)
    out["mask"] = words[req, i]
    out["positions"] = (ctx[req] + seen.view(R, n, -1).sum(-1)[req, i] - 1).int()
    return out


def _plain_write(s):
    P = s["c"]["P"]
    page, off = s["slots"].long() // P, s["slots"].long() % P
    s["k"][page, :, off] = s["kv"][:, 0]
    s["v"][page, :, off] = s["kv"][:, 1]
    return {"k": s["k"], "v": s["v"]}


def _plain_attend(s):
    c, T = s["c"], s["T"]
    R, n, P, D, G = c["R"], c["n"], c["P"], c["D"], c["hq"] // c["hkv"]
    ctx, start = s["ctx"].long(), s["start"].long()
    L = s["table"].shape[1] * P
    pages = s["table"].long().clamp(min=0)
    k, v = (s[x][pages].transpose(1, 2).reshape(R, c["hkv"], L, D).float() for x in ("k", "v"))
    i = torch.arange(n, device=DEV)
    tok = (start[:-1, None] + i).clamp(max=T - 1)
    q = s["q"].float()[tok].view(R, n, c["hkv"], G, D).transpose(1, 2).reshape(R, c["hkv"], n * G, D)
    x = torch.matmul(q, k.transpose(2, 3)) * (D ** -0.5)
    j = torch.arange(L, device=DEV) - ctx[:, None]          # place among the new tokens
    if s["mask"] is None:
        own_part = (j[:, None, :] <= i[None, :, None])
    else:
        word = (j.clamp(min=0) >> 6).clamp(max=s["mask"].shape[1] - 1)
        bits = torch.gather(s["mask"][tok], 2, word[:, None, :].expand(R, n, L))
        own_part = ((bits >> (j.clamp(min=0) & 63)[:, None, :]) & 1).bool()
    seen = (j < 0)[:, None, :] | (own_part & (j < (start[1:] - start[:-1])[:, None])[:, None, :])
    x = x.view(R, c["hkv"], n, G, L).masked_fill(~seen[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    o = torch.matmul(p.view(R, c["hkv"], n * G, L), v).view(R, c["hkv"], n, G, D)
    o = o / p.sum(-1, keepdim=True).clamp(min=1e-30)
    req, t = _request_of(start, T, R)
    return o.permute(0, 2, 1, 3, 4)[req, t - start[req]].reshape(T, c["hq"], D).bfloat16()


def _plain_accept(s):
    c, P = s["c"], s["c"]["P"]
    ctx, lens, paths = s["ctx"].long(), s["lens"].long(), s["paths"].long()
    i = torch.arange(paths.shape[1], device=DEV)
    taken = i[None, :] < lens[:, None]
    src = ctx[:, None] + torch.where(taken, paths, i)
    dst = ctx[:, None] + i
    last = s["table"].shape[1] - 1

    def place(x):  # rows past a request's pages stand for its row 0, in both places
        page = torch.gather(s["table"].long(), 1, (x // P).clamp(max=last))
        bad = (page < 0) | (x // P > last) | ~taken
        return torch.where(bad, s["table"][:, :1].long(), page), torch.where(bad, 0, x % P)

    (sp, so), (dp, do) = place(src), place(dst)
    for cache in (s["k"], s["v"]):
        cache[:, dp, :, do] = cache[:, sp, :, so]
    return {"k": s["k"], "v": s["v"], "ctx": (ctx + lens).int()}


def run(state):
    s, op = state, state["c"]["op"]
    if not own:
        return {"plan": _plain_plan, "write": _plain_write, "attend": _plain_attend,
                "accept": _plain_accept}[op](s)
    import gemm_swiglu_mlp_gb300 as sg
    if op == "plan":
        p = s["plan"] = sg.swiglu_cache_plan(
            s["ctx"], s["new"], s["held"], s["table"], s["free"], s["c"]["P"], s["T"],
            parents=s["parents"], out=s["plan"])
        out = {"table": s["table"], "start": p.query_start, "slots": p.slots,
               "held": p.pages_held, "counts": p.counts, "positions": p.positions}
        return out if p.mask is None else {**out, "mask": p.mask}
    if op == "write":
        sg.swiglu_cache_write(s["kv"][:, 0], s["kv"][:, 1], s["slots"], s["k"], s["v"])
        return {"k": s["k"], "v": s["v"]}
    if op == "attend":
        return sg.swiglu_tree_attention(s["q"], s["k"], s["v"], s["table"], s["ctx"], s["start"],
                                        mask=s["mask"])
    new_ctx = sg.swiglu_cache_accept(s["k"], s["v"], s["table"], s["ctx"], s["paths"], s["lens"])
    return {"k": s["k"], "v": s["v"], "ctx": new_ctx}


# ----------------------------------------------------------------- what a pass needs
def work(case):
    c = dict(case)
    ctx, new = _lengths(c)
    T, R = int(new.sum()), c["R"]
    if c["op"] == "plan":
        fresh = (ctx + new + c["P"] - 1) // c["P"] - (ctx + c["P"] - 1) // c["P"]
        words = (c["n"] + 63) // 64 if c["tree"] else 0
        # lengths, held pages and parents in; slots, positions, masks and new pages out
        return {"bytes": 4 * (5 * R + 1 + 3) + 8 * T + 12 * int(fresh.sum())
                + (4 * T + 8 * words * T if c["tree"] else 0), "flops": 0}
    row = 2 * c["hkv"] * c["D"]
    if c["op"] == "write":
        return {"bytes": 4 * T * row + 4 * T, "flops": 0}
    if c["op"] == "accept":
        depth = max(2, min(6, c["n"] // 4))
        moved = 0.0  # rows that move, on average over the paths that prepare() draws
        for i in range(R):
            top = min(depth, max(1, int(new[i]) // 2))
            moved += sum((p - 1) / 2 for p in range(1, top + 1)) / top
        return {"bytes": 4 * moved * c["layers"] * row + 4 * R * (depth + 3), "flops": 0}
    seen = int((new * (ctx + (new + 1) / 2)).sum())       # query-key pairs of the context and half of the new
    return {"bytes": 2 * int((ctx + new).sum()) * row + 4 * T * c["hq"] * c["D"],
            "flops": 4 * seen * c["hq"] * c["D"]}


# ----------------------------------------------------------------- 64-bit results
def _exact_attend(s):
    c = s["c"]
    P, D, G = c["P"], c["D"], c["hq"] // c["hkv"]
    ctx, start, table = s["ctx"].tolist(), s["start"].tolist(), s["table"].tolist()
    out = torch.zeros(s["T"], c["hq"], D, dtype=torch.float64, device=DEV)
    words = None if s["mask"] is None else s["mask"].cpu().numpy().view(np.uint64)
    for r in range(c["R"]):
        t0, t1 = start[r], start[r + 1]
        n, L = t1 - t0, ctx[r] + t1 - t0
        if words is None:
            vis = np.tril(np.ones((n, n), bool))
        else:
            j = np.arange(n, dtype=np.uint64)
            vis = (words[t0:t1][:, (j >> np.uint64(6)).astype(int)] >> (j & np.uint64(63))) & np.uint64(1)
        vis = torch.from_numpy(np.ascontiguousarray(vis.astype(bool))).to(DEV)
        used = table[r][: -(-L // P)]
        for h in range(c["hkv"]):
            k = s["k"][used, h].reshape(-1, D)[:L].double()
            v = s["v"][used, h].reshape(-1, D)[:L].double()
            for a in range(0, n, 64):
                b = min(n, a + 64)
                q = s["q"][t0 + a:t0 + b, h * G:(h + 1) * G].double()
                x = torch.einsum("tgd,ld->tgl", q, k) / math.sqrt(D)
                x[:, :, ctx[r]:] = x[:, :, ctx[r]:].masked_fill(~vis[a:b, None, :], -math.inf)
                out[t0 + a:t0 + b, h * G:(h + 1) * G] = torch.einsum(
                    "tgl,ld->tgd", torch.softmax(x, -1), v)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c, P = s["c"], s["c"]["P"]
    if c["op"] == "plan":
        return None
    if c["op"] == "attend":
        return _exact_attend(s)
    table, ctx = s["table"].cpu().numpy(), s["ctx"].cpu().numpy()
    if c["op"] == "write":
        slots = s["slots"].cpu().numpy()
        for which, cache in ((0, s["k"]), (1, s["v"])):
            flat = cache.transpose(1, 2).reshape(-1, c["hkv"], c["D"]).clone()
            flat[torch.from_numpy(slots.astype(np.int64)).to(DEV)] = s["kv"][:, which]
            s["k" if which == 0 else "v"] = flat.view(-1, P, c["hkv"], c["D"]).transpose(1, 2)
        return {"k": s["k"].contiguous().double(), "v": s["v"].contiguous().double()}
    paths, lens = s["paths"].cpu().numpy(), s["lens"].cpu().numpy()
    for name in ("k", "v"):
        before = s[name].clone()
        for r in range(c["R"]):
            for i in range(lens[r]):
                a, b = ctx[r] + paths[r, i], ctx[r] + i
                s[name][:, table[r, b // P], :, b % P] = before[:, table[r, a // P], :, a % P]
    return {"k": s["k"].double(), "v": s["v"].double(), "ctx": None}
