"""The paged-cache operators on the GPU against their 64-bit definitions:
whole numbers and copies exactly, attention within the bound of BF16 weights
and one BF16 rounding (cache_ref.attend)."""
import numpy as np
import pytest

from tests import cache_ref as ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gemm_swiglu_mlp_gb300 import build
    build.build()
    import gemm_swiglu_mlp_gb300 as mod
    torch.cuda.set_device(0)
    return mod


def dev_i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def dev_i64(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int64)).cuda()


def dev_bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits, np.uint16).view(np.int16)).cuda().view(
        torch.bfloat16)


def host_bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


# ------------------------------------------------------------------ plan
def run_plan(sg, ctx, new, held, table, free, P, max_tokens, parents=None, head=0, out=None):
    tab = dev_i32(table)
    got = sg.swiglu_cache_plan(dev_i32(ctx), dev_i32(new), dev_i32(held), tab, dev_i32(free), P,
                               max_tokens, parents=None if parents is None else dev_i32(parents),
                               free_head=dev_i32([head]) if head else None, out=out)
    want = ref.plan(ctx, new, held, np.array(table, np.int64), free, P, max_tokens, parents, head)
    for name in ("query_start", "slots", "positions", "pages_held", "counts"):
        assert np.array_equal(getattr(got, name).cpu().numpy(), want[name]), name
    assert np.array_equal(tab.cpu().numpy(), want["table"])
    if parents is not None:
        assert np.array_equal(got.mask.cpu().numpy(), want["mask"])
    return got


@pytest.mark.parametrize("R,n,width,P,extra,short,head", [
    (1, 1, 0, 16, 0, 0, 0),          # one token
    (1, 0, 0, 16, 0, 0, 0),          # nothing new
    (5, 9, 9, 16, 3, 0, 4),          # trees, tokens past the end, a moved free list
    (33, 70, 70, 32, 0, 0, 0),       # two mask words
    (17, 130, 130, 64, 5, 0, 2),     # three
    (700, 3, 3, 16, 1, 0, 0),        # more requests than threads
    (40, 50, 0, 128, -30, 0, 0),     # chains; fewer rows than tokens
    (12, 40, 40, 16, 0, 9, 0),       # the free list runs out
    (3, 20000, 0, 16, 0, 0, 0),      # prompts
])
def test_plan(sg, R, n, width, P, extra, short, head):
    rng = np.random.default_rng(R * 1000 + n)
    ctx = rng.integers(0, 6 * P, R)
    new = rng.integers(0, n + 1, R)
    new[0] = n
    held = -(-ctx // P) + rng.integers(0, 3, R) * (rng.random(R) < 0.3)
    parents = None
    if width:
        parents = np.stack([ref.random_parents(rng, width) for _ in range(R)])
    max_pages = int((-(-(ctx + new) // P)).max()) + 3
    table = np.full((R, max_pages), -1, np.int64)
    pages = rng.permutation(int(held.sum()) + 10)
    at = 0
    for r in range(R):
        held[r] = min(held[r], max_pages)
        table[r, :held[r]] = pages[at:at + held[r]]
        at += held[r]
    need = int(np.maximum(-(-(ctx + new) // P) - held, 0).sum())
    free = rng.permutation(need + head - short + 2 * (short == 0)) + 100000
    run_plan(sg, ctx, new, held, table, free, P, max(int(new.sum()) + extra, 0), parents, head)


def test_plan_odd_inputs(sg):
    # negative lengths count as none; a table too short for the context; parents
    # that are no earlier token hang on the context; more new tokens than columns
    par = np.array([[5, 0, 1, 3], [-1, -7, 1, 2], [-1, 0, 1, 2]], np.int32)
    run_plan(sg, [-3, 40, 90], [4, 9, 2], [-1, 2, 9], np.arange(15).reshape(3, 5), [50, 51, 52, 53],
             16, 12, par)


def test_plan_no_requests_and_reused_buffers(sg):
    z = np.zeros(0, np.int32)
    got = run_plan(sg, z, z, z, np.zeros((0, 4)), [1, 2], 16, 3)
    assert got.slots.tolist() == [-1, -1, -1]
    first = run_plan(sg, [5], [2], [1], [[3, -1]], [8], 16, 4)
    again = run_plan(sg, [15], [3], [1], [[3, -1]], [8], 16, 4, out=first)
    assert again.slots.data_ptr() == first.slots.data_ptr()


# ------------------------------------------------------------------ write
@pytest.mark.parametrize("T,H,D,P,fused", [
    (1, 1, 64, 16, False), (7, 2, 128, 16, True), (65, 4, 128, 32, True), (333, 8, 64, 64, False),
    (50, 3, 128, 128, True), (9, 40, 64, 16, True), (4099, 1, 128, 16, False)])
def test_write(sg, T, H, D, P, fused):
    rng = np.random.default_rng(T + H)
    pages = -(-T // P) + 3
    kc, vc = (rng.integers(0, 1 << 16, (pages, H, P, D)).astype(np.uint16) for _ in range(2))
    kv = rng.integers(0, 1 << 16, (T, 2, H, D)).astype(np.uint16)
    slots = rng.permutation(pages * P)[:T].astype(np.int64)
    slots[rng.random(T) < 0.1] = -1
    if T > 5:
        slots[3], slots[4] = pages * P, (1 << 31) - 1      # no such rows
    kct, vct, t = dev_bf16(kc), dev_bf16(vc), dev_bf16(kv)
    k, v = t[:, 0], t[:, 1]
    if not fused:
        k, v = k.contiguous(), v.transpose(0, 1).contiguous().transpose(0, 1)   # heads outermost
    sg.swiglu_cache_write(k, v, dev_i32(slots), kct, vct)
    for i, s in enumerate(slots):
        if 0 <= s < pages * P:
            kc[s // P, :, s % P], vc[s // P, :, s % P] = kv[i, 0], kv[i, 1]
    assert np.array_equal(host_bits(kct), kc) and np.array_equal(host_bits(vct), vc)


def test_write_nothing(sg):
    c = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    e = torch.zeros(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    sg.swiglu_cache_write(e, e, dev_i32([]), c, c.clone())


# ------------------------------------------------------------------ accept
@pytest.mark.parametrize("R,n,width,layers,H,D,P", [
    (1, 4, 3, 1, 1, 64, 16), (6, 20, 7, 3, 2, 128, 16), (3, 64, 12, 2, 3, 64, 32),
    (2, 200, 80, 2, 1, 128, 16), (40, 9, 5, 1, 8, 128, 64)])
def test_accept(sg, R, n, width, layers, H, D, P):
    rng = np.random.default_rng(R + n)
    ctx = rng.integers(0, 3 * P, R)
    ctx[0] = 0
    need = -(-(ctx + n) // P)
    pages = int(need.sum()) + 2
    table = ref.tables(rng, need, pages)
    shape = (layers, pages, H, P, D)
    caches = [rng.integers(0, 1 << 16, shape).astype(np.uint16) for _ in range(2)]
    # increasing paths, also ones whose rows are each other's targets
    lens = rng.integers(0, width + 1, R)
    lens[0] = width
    paths = np.full((R, width), -1, np.int64)
    for r in range(R):
        top = int(rng.integers(lens[r], n + 1))
        paths[r, :lens[r]] = np.sort(rng.choice(top, lens[r], replace=False)) if lens[r] else []
    paths[0, :] = np.arange(width) + 1       # every row from its neighbour
    want = ref.accept(caches, table, ctx, paths, lens, P)
    k, v = dev_bf16(caches[0]), dev_bf16(caches[1])
    if layers == 1:
        k, v = k[0], v[0]
    new = sg.swiglu_cache_accept(k, v, dev_i32(table), dev_i32(ctx), dev_i32(paths), dev_i32(lens))
    assert np.array_equal(new.cpu().numpy(), ctx + lens)
    assert np.array_equal(host_bits(k).reshape(shape), want[0])
    assert np.array_equal(host_bits(v).reshape(shape), want[1])


def test_accept_without_pages_or_requests(sg):
    k = torch.randn(3, 1, 16, 64, device="cuda").bfloat16()
    v = k.clone()
    keep = host_bits(k)
    # the source's page is missing; its number is outside the cache; path longer than the table
    table = dev_i32([[0, -1], [1, 99], [2, -1]])
    new = sg.swiglu_cache_accept(k, v, table, dev_i32([10, 10, 31]), dev_i32([[9], [9], [5]]),
                                 dev_i32([1, 1, 4]))
    assert new.tolist() == [11, 11, 32]
    assert np.array_equal(host_bits(k), keep) and np.array_equal(host_bits(v), keep)
    e = dev_i32([])
    assert sg.swiglu_cache_accept(k, v, e.view(0, 1), e, e.view(0, 1), e).numel() == 0


# ------------------------------------------------------------------ attention
class Case:
    """Inputs of one step: random rows where a position is in use, NaN in every
    other row of the cache."""

    def __init__(self, seed, ctx, new, Hq, Hkv, D, P, tree, qscale=1.5, words=None, extra_rows=0):
        rng = self.rng = np.random.default_rng(seed)
        self.ctx, self.new = np.array(ctx), np.array(new)
        self.Hq, self.Hkv, self.D, self.P = Hq, Hkv, D, P
        R = len(ctx)
        self.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        self.T = int(self.start[-1]) + extra_rows
        need = -(-(self.ctx + self.new) // P)
        pages = int(need.sum()) + 3
        self.table = ref.tables(rng, need, pages)
        self.k = np.full((pages, Hkv, P, D), 0x7FC0, np.uint16)
        self.v = self.k.copy()
        for r in range(R):
            x = np.arange(self.ctx[r] + self.new[r])
            for c in (self.k, self.v):
                c[self.table[r, x // P], :, x % P] = ref.f32_to_bits(
                    rng.standard_normal((len(x), Hkv, D)))
        self.q = ref.f32_to_bits(qscale * rng.standard_normal((self.T, Hq, D)))
        if tree:
            self.visible = [ref.ancestors(ref.random_parents(rng, n), n) for n in self.new]
            self.words = words or max(1, -(-int(max(new, default=1)) // 64))
        else:
            self.visible = [np.tril(np.ones((n, n), bool)) for n in self.new]
            self.words = 0

    def mask(self):
        if not self.words:
            return None
        m = np.zeros((self.T, self.words), np.int64)
        for r, seen in enumerate(self.visible):
            m[self.start[r]:self.start[r + 1]] = ref.pack_words(seen, self.words)
        return m

    def row(self, r, x):
        return self.table[r, x // self.P], slice(None), x % self.P

    def run(self, sg, scale=None, q=None, **kw):
        m = self.mask()
        self.last = sg.swiglu_tree_attention(
            dev_bf16(self.q) if q is None else q, dev_bf16(self.k), dev_bf16(self.v),
            dev_i32(self.table), dev_i32(self.ctx), dev_i32(self.start),
            mask=None if m is None else dev_i64(m), scale=scale, **kw)
        assert sg.swiglu_check_device_status() == 0
        return host_bits(self.last)

    def check(self, got, scale=None):
        scale = self.D ** -0.5 if scale is None else scale
        want, bound = ref.attend(ref.bits_to_f64(self.q), ref.bits_to_f64(self.k),
                                 ref.bits_to_f64(self.v), self.table, self.ctx, self.start,
                                 self.visible, scale, self.P)
        g = ref.bits_to_f64(got)
        both = np.isfinite(want)
        assert np.array_equal(np.isnan(g), np.isnan(want))
        assert np.array_equal(g[~both & ~np.isnan(want)], want[~both & ~np.isnan(want)])
        over = np.abs(g - want)[both] - bound[both]
        assert over.size == 0 or over.max() <= 0, (over.max(), int((over > 0).sum()))


SHAPES = [(7, 1, 64, 16), (12, 2, 128, 32), (8, 8, 64, 64), (14, 2, 128, 16), (16, 1, 128, 128)]


@pytest.mark.parametrize("Hq,Hkv,D,P", SHAPES)
@pytest.mark.parametrize("tree", [False, True])
def test_attention_lengths_around_tiles(sg, Hq, Hkv, D, P, tree):
    """Contexts that end just before, on and after pages and blocks of 128
    positions, with one to nine new tokens."""
    ctx = [0, 1, 15, 16, 17, 119, 126, 127, 128, 129, 250, 255, 256, 257, 384]
    new = [1, 1, 2, 1, 5, 9, 2, 1, 1, 3, 9, 2, 1, 7, 1]
    c = Case(Hq * D + P, ctx, new, Hq, Hkv, D, P, tree)
    c.check(c.run(sg))


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,P", [
    ([300, 70], [18, 19], 7, 1, 128, 16),      # 126 and 133 rows of one head
    ([40, 500], [36, 37], 14, 2, 128, 16),     # 252 and 259
    ([200], [64], 8, 1, 64, 64),               # 512 rows
    ([100, 3], [130, 65], 4, 2, 64, 16),       # more than one mask word
    ([0, 640], [128, 129], 2, 2, 128, 32),     # no context; blocks of hidden new tokens
    ([33], [300], 1, 1, 64, 16),
    ([60, 61], [3, 2], 128, 1, 64, 16),        # as many heads as a tile has rows
    ([20], [5], 96, 1, 128, 16),
])
@pytest.mark.parametrize("tree", [False, True])
def test_attention_many_rows(sg, ctx, new, Hq, Hkv, D, P, tree):
    c = Case(sum(ctx) + Hq, ctx, new, Hq, Hkv, D, P, tree)
    c.check(c.run(sg))


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,P,tree", [
    ([9000], [1], 7, 1, 128, 16, False),
    ([9001], [25], 5, 1, 64, 64, True),
    ([5000, 12, 7003], [40, 1, 30], 14, 2, 128, 32, True),
    ([4100], [70], 8, 2, 128, 16, False),
    ([20011], [3], 2, 2, 64, 128, True),
])
def test_attention_long_contexts(sg, ctx, new, Hq, Hkv, D, P, tree):
    """Few requests and long contexts: the work of one head is shared."""
    c = Case(sum(ctx), ctx, new, Hq, Hkv, D, P, tree)
    c.check(c.run(sg))


@pytest.mark.parametrize("D,P", [(128, 16), (64, 32)])
@pytest.mark.parametrize("tree", [False, True])
def test_attention_items_of_two_to_many_blocks(sg, D, P, tree):
    """One long line of work: items of one, two, some and many blocks, of a few
    rows, one row tile and two, in both forms."""
    ctx = [300, 6000, 900, 50, 1500, 2500, 100, 4000, 0, 3000]
    new = [1, 3, 20, 40, 2, 33, 9, 1, 5, 64]
    c = Case(D + tree, ctx, new, 8, 1, D, P, tree)
    c.check(c.run(sg))
    c = Case(D + tree + 2, ctx[::-1], new, 7, 1, D, P, tree)
    c.check(c.run(sg))


def test_attention_many_requests(sg):
    rng = np.random.default_rng(5)
    new = rng.integers(0, 4, 300)
    c = Case(6, rng.integers(0, 200, 300), new, 4, 2, 64, 16, True)
    c.check(c.run(sg))
    c = Case(7, rng.integers(0, 400, 37), rng.integers(0, 30, 37), 12, 2, 128, 32, False)
    c.check(c.run(sg))


def test_attention_rows_that_see_nothing(sg):
    """Empty mask rows, requests without new tokens, rows past the last
    request, and mask words that end before the tree does."""
    c = Case(8, [0, 0, 30, 0, 5], [3, 0, 4, 70, 2], 7, 1, 128, 16, True, words=1, extra_rows=5)
    c.visible[0][:] = False
    c.visible[0][1, 0] = True
    c.visible[2][:] = False            # these still see their context
    c.visible[3][:, 64:] = False       # past the only word
    c.visible[3][65] = False
    got = c.run(sg)
    c.check(got)
    assert not got[c.start[-1]:].any() and not got[0].any() and not got[2].any()


def test_attention_scores_of_every_size(sg):
    """Large scores (one position takes all), a scale of its own, and scores
    that are all -inf."""
    for seed, qscale, scale in ((9, 40.0, None), (10, 1.0, 3.0), (11, 1.0, 1e-6)):
        c = Case(seed, [100, 300], [5, 9], 8, 2, 128, 16, True, qscale=qscale)
        c.check(c.run(sg, scale=scale), scale=scale)
    # rising scores: the running maximum moves at every block
    c = Case(12, [1500], [4], 6, 1, 64, 16, False)
    x = np.arange(1504)
    c.q[:] = ref.f32_to_bits(np.ones(1))[0]
    c.k[c.table[0, x // 16], :, x % 16] = ref.f32_to_bits(0.2 * (x[:, None, None] // 40) *
                                                         np.ones((1, 1, 64)))
    c.check(c.run(sg))
    c.k[c.table[0, x // 16], :, x % 16] = 0xFF80       # -inf keys against positive queries
    got = c.run(sg)
    assert not got.any()


@pytest.mark.parametrize("bad", [0x7FC0, 0x7F80, 0xFF80])
@pytest.mark.parametrize("where", ["k", "v"])
def test_attention_hidden_values_stay_hidden(sg, bad, where):
    """NaN and Inf in the rows of new tokens that others do not see: only the
    rows that see them are touched."""
    for tree, new in ((True, [9, 40, 3]), (False, [9, 140, 3])):
        c = Case(13, [125, 100, 0], new, 7, 1, 128, 16, tree)
        for r, j in ((0, 4), (1, 0 if tree else 27), (1, 31), (2, 2)):
            getattr(c, where)[c.row(r, c.ctx[r] + j)] = bad
        if where == "k":
            c.q = np.where(c.q & 0x7FFF == 0, np.uint16(0x3F80), c.q)
        c.check(c.run(sg))


def test_attention_visible_infinities(sg):
    """Inf and NaN in values of the context reach every row that sees them."""
    c = Case(14, [200, 20], [6, 3], 4, 2, 64, 16, True)
    c.v[c.row(0, 150)][:, 5] = 0x7F80
    c.v[c.row(0, 17)][:, 9] = 0x7FC0
    c.v[c.row(1, 19)][:, 0] = 0xFF80
    c.check(c.run(sg))


def test_attention_strides_out_and_workspace(sg):
    c = Case(15, [100, 900], [4, 8], 12, 2, 128, 16, True)
    whole = torch.randn(c.T, 3, 12, 128, device="cuda").bfloat16()
    whole[:, 1] = dev_bf16(c.q)
    out = torch.full((c.T, 12, 128), float("nan"), device="cuda", dtype=torch.bfloat16)
    need = sg.swiglu_tree_attention_workspace_bytes(c.T, 12, 2, 128)
    ws = torch.zeros(max(need, 256), dtype=torch.uint8, device="cuda")
    got = c.run(sg, q=whole[:, 1], out=out, workspace=ws)
    assert c.last.data_ptr() == out.data_ptr()
    c.check(got)
    by_head = dev_bf16(c.q).transpose(0, 1).contiguous().transpose(0, 1)
    assert np.array_equal(c.run(sg, q=by_head, workspace=ws), got)     # and bit for bit again


def test_results_belong_to_the_given_stream(sg):
    """A block that the current stream has freed, but still reads, is not handed
    to a result that another stream writes at once."""
    ctx = torch.full((64,), 5, dtype=torch.int32, device="cuda")
    table = torch.zeros(64, 1, dtype=torch.int32, device="cuda")
    k, v = torch.zeros(2, 1, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    paths = torch.zeros(64, 1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(64, dtype=torch.int32, device="cuda")
    q = torch.zeros(64, 1, 64, dtype=torch.bfloat16, device="cuda")
    start = torch.arange(65, dtype=torch.int32, device="cuda")
    free = torch.zeros(1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    calls = [lambda: sg.swiglu_cache_accept(k, v, table, ctx, paths, lens, stream=side),
             lambda: sg.swiglu_tree_attention(q, k, v, table, ctx, start, stream=side),
             lambda: sg.swiglu_cache_plan(ctx, lens, torch.ones_like(ctx), table, free, 16, 64,
                                          stream=side).slots]
    for call in calls:
        got = call()
        size = (got.numel(), got.dtype)
        side.synchronize()
        del got
        old = torch.empty(size[0], dtype=size[1], device="cuda")   # of the current stream
        where = old.data_ptr()
        del old
        assert call().data_ptr() != where
        side.synchronize()



def test_attention_other_stream_and_graph(sg):
    """Calls on a side stream, and a captured step replayed with other lengths."""
    c = Case(16, [700, 30, 2000], [9, 1, 12], 7, 1, 128, 16, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q, k, v, mask = dev_bf16(c.q), dev_bf16(c.k), dev_bf16(c.v), dev_i64(c.mask())
    table, ctx, start = dev_i32(c.table), dev_i32(c.ctx), dev_i32(c.start)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        a = sg.swiglu_tree_attention(q, k, v, table, ctx, start, mask=mask)
    b = sg.swiglu_tree_attention(q, k, v, table, ctx, start, mask=mask, stream=side)
    side.synchronize()
    c.check(host_bits(a))
    assert torch.equal(a, b)
    ws = torch.zeros(max(256, sg.swiglu_tree_attention_workspace_bytes(c.T, 7, 1, 128)),
                     dtype=torch.uint8, device="cuda")
    out = torch.empty_like(a)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sg.swiglu_tree_attention(q, k, v, table, ctx, start, mask=mask, out=out, workspace=ws)
    for ctx2 in (c.ctx, np.array([650, 31, 3]), np.array([0, 0, 0])):
        c.ctx = ctx2
        ctx.copy_(dev_i32(ctx2))
        # the new tokens' rows at their new places
        for r in range(3):
            for i in range(int(c.new[r])):
                for cache in (c.k, c.v):
                    cache[c.row(r, ctx2[r] + i)] = ref.f32_to_bits(
                        c.rng.standard_normal((1, 128)))
        k.copy_(dev_bf16(c.k))
        v.copy_(dev_bf16(c.v))
        g.replay()
        torch.cuda.synchronize()
        c.check(host_bits(out))


def test_attention_nothing_to_do(sg):
    c = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.ones(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    out = sg.swiglu_tree_attention(q, c, c.clone(), dev_i32([[0]]), dev_i32([3]), dev_i32([0, 0]))
    assert out.shape == (0, 2, 64)
    q = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    out = sg.swiglu_tree_attention(q, c, c.clone(), dev_i32(np.zeros((0, 1))), dev_i32([]),
                                   dev_i32([0]))
    assert not out.any()


def test_attention_table_entries_outside_the_cache(sg):
    """Entries of the table that name no page are never followed."""
    c = Case(17, [60, 20], [3, 2], 4, 2, 64, 16, False)
    q, k, v = dev_bf16(c.q), dev_bf16(c.k), dev_bf16(c.v)
    for wrong in (-1, len(c.k), (1 << 31) - 1, -(1 << 31)):
        table = c.table.copy()
        table[0, 1] = wrong
        got = sg.swiglu_tree_attention(q, k, v, dev_i32(table), dev_i32(c.ctx), dev_i32(c.start))
        sg.swiglu_check_device_status()
        # the other request is not touched by it
        keep = c.visible, c.ctx
        want, bound = ref.attend(ref.bits_to_f64(c.q), ref.bits_to_f64(c.k), ref.bits_to_f64(c.v),
                                 c.table, c.ctx, c.start, c.visible, 64 ** -0.5, 16)
        assert keep is not None
        diff = np.abs(ref.bits_to_f64(host_bits(got)) - want)[3:]
        assert (diff <= bound[3:]).all()


@pytest.mark.parametrize("D", [64, 128])
def test_cache_past_32_bit_offsets(sg, D):
    """Pages whose offsets pass 2^32 elements: written, moved and read."""
    H, P = 2, 128
    pages = (1 << 32) // (H * P * D) + 4
    k = torch.empty(pages, H, P, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty(pages, H, P, D, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(18)
    table = np.array([[pages - 1, pages - 3, 1]], np.int32)
    x = np.arange(300)
    rows = ref.f32_to_bits(rng.standard_normal((300, 2, H, D)))
    kv = dev_bf16(rows)
    slots = table[0, x // P].astype(np.int64) * P + x % P
    sg.swiglu_cache_write(kv[:, 0], kv[:, 1], dev_i32(slots), k, v)
    # positions 200 + (0, 3, 9) become 200, 201, 202
    new = sg.swiglu_cache_accept(k, v, dev_i32(table), dev_i32([200]), dev_i32([[0, 3, 9]]),
                                 dev_i32([3]))
    assert new.tolist() == [203]
    rows[201], rows[202] = rows[203].copy(), rows[209].copy()
    q = ref.f32_to_bits(rng.standard_normal((4, 4, D)))
    got = sg.swiglu_tree_attention(dev_bf16(q), k, v, dev_i32(table), dev_i32([296]),
                                   dev_i32([0, 4]))
    kk, vv = (np.zeros((3, H, P, D)) for _ in range(2))
    kk[x // P, :, x % P] = ref.bits_to_f64(rows[:, 0])
    vv[x // P, :, x % P] = ref.bits_to_f64(rows[:, 1])
    want, bound = ref.attend(ref.bits_to_f64(q), kk, vv, np.array([[0, 1, 2]]), [296], [0, 4],
                             [np.tril(np.ones((4, 4), bool))], D ** -0.5, P)
    assert (np.abs(ref.bits_to_f64(host_bits(got)) - want) <= bound).all()


def test_step_end_to_end(sg):
    """plan, write, attend and accept as one step after another: the tokens that
    are accepted are the context of the next step."""
    rng = np.random.default_rng(19)
    R, Hq, H, D, P, width = 5, 6, 2, 64, 16, 9
    pages = 64
    k = torch.full((pages, H, P, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    table, free = dev_i32(np.full((R, 8), -1)), dev_i32(rng.permutation(pages))
    ctx, held, head = dev_i32(np.zeros(R)), dev_i32(np.zeros(R)), dev_i32([0])
    seqs = [np.zeros((0, 2, H, D), np.uint16) for _ in range(R)]    # the oracle's contexts
    for step in range(6):
        new = rng.integers(1, width + 1, R)
        T = int(new.sum())
        par = np.stack([ref.random_parents(rng, width) for _ in range(R)])
        plan = sg.swiglu_cache_plan(ctx, dev_i32(new), held, table, free, P, T + 2,
                                    parents=dev_i32(par), free_head=head)
        kv = ref.f32_to_bits(rng.standard_normal((T + 2, 2, H, D)))
        q = ref.f32_to_bits(rng.standard_normal((T + 2, Hq, D)))
        t = dev_bf16(kv)
        sg.swiglu_cache_write(t[:, 0], t[:, 1], plan.slots, k, v)
        out = sg.swiglu_tree_attention(dev_bf16(q), k, v, table, ctx, plan.query_start,
                                       mask=plan.mask)
        # the oracle: each request's rows in a cache of its own
        start = np.concatenate([[0], np.cumsum(new)])
        lens, paths = np.zeros(R, np.int64), np.zeros((R, width), np.int64)
        for r in range(R):
            rows = np.concatenate([seqs[r], kv[start[r]:start[r + 1]]])
            L = len(rows)
            one = np.zeros((-(-L // P), 2, H, P, D))
            one[np.arange(L) // P, :, :, np.arange(L) % P] = ref.bits_to_f64(rows)
            seen = ref.ancestors(par[r], int(new[r]))
            want, bound = ref.attend(ref.bits_to_f64(q[start[r]:start[r + 1]]), one[:, 0], one[:, 1],
                                     np.arange(len(one))[None], [len(seqs[r])], [0, new[r]], [seen],
                                     D ** -0.5, P)
            got = ref.bits_to_f64(host_bits(out))[start[r]:start[r + 1]]
            assert (np.abs(got - want) <= bound).all(), (step, r)
            leaf = int(rng.integers(0, new[r]))
            path = np.nonzero(seen[leaf])[0]
            lens[r] = len(path)
            paths[r, :len(path)] = path
            seqs[r] = np.concatenate([seqs[r], kv[start[r] + path]])
        ctx = sg.swiglu_cache_accept(k, v, table, ctx, dev_i32(paths), dev_i32(lens))
        held, head = plan.pages_held, plan.counts[2:3]
        assert ctx.tolist() == [len(s) for s in seqs]
    sg.swiglu_check_device_status()
