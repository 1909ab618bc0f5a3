"""The paged-cache entry points without a GPU: their reference by hand, and
the refusals made on the host before anything is launched."""
import numpy as np
import pytest

from tests import cache_ref

P16 = 0x10000        # fake, aligned "device" addresses: never dereferenced


@pytest.fixture(scope="module")
def lib():
    from gemm_swiglu_mlp_gb300 import build
    build.build()
    import gemm_swiglu_mlp_gb300 as sg
    return sg.load_library()


def _addr(i):
    return P16 + i * 0x10000000


def test_plan_reference_by_hand():
    # two requests, page size 4: the first has 5 of 8 rows of 2 pages and adds
    # a tree of 4 (one new page), the second starts with 1 token
    table = np.array([[7, 3, -1], [-1, -1, -1]], np.int32)
    par = np.array([[-1, 0, 0, 2], [-1, -1, -1, -1]], np.int32)
    out = cache_ref.plan([5, 0], [4, 1], [2, 0], table, [9, 8], 4, 6, par)
    assert out["query_start"].tolist() == [0, 4, 5]
    assert table.tolist() == [[7, 3, 9], [8, -1, -1]]
    assert out["slots"].tolist() == [13, 14, 15, 36, 32, -1]
    assert out["positions"].tolist() == [5, 6, 6, 7, 0, 0]
    assert out["mask"][:, 0].tolist() == [1, 3, 5, 13, 1, 0]
    assert out["pages_held"].tolist() == [3, 1] and out["counts"].tolist() == [5, 2, 2]


def test_attend_reference_by_hand():
    # one head of size 1, two context rows and a hidden NaN: equal scores
    k = np.zeros((1, 1, 4, 1))
    v = np.array([1.0, 3.0, np.nan, 8.0]).reshape(1, 1, 4, 1)
    q = np.ones((2, 1, 1))
    vis = [np.array([[False, False], [False, True]])]
    out, _ = cache_ref.attend(q, k, v, np.zeros((1, 1), np.int64), [2], [0, 2], vis, 1.0, 4)
    assert out[:, 0, 0].tolist() == [2.0, 4.0]


def test_plan_refusals(lib):
    a = [_addr(i) for i in range(12)]
    ok = dict(ctx=a[0], new=a[1], held=a[2], table=a[3], R=4, pages=8, free=a[4], nfree=4,
              head=None, P=16, par=a[5], width=8, T=16, start=a[6], slots=a[7], pos=a[8],
              heldo=a[9], counts=a[10], mask=a[11])

    def call(**kw):
        x = dict(ok, **kw)
        return lib.swiglu_cache_plan(
            x["ctx"], x["new"], x["held"], x["table"], x["R"], x["pages"], x["free"], x["nfree"],
            x["head"], x["P"], x["par"], x["width"], x["T"], x["start"], x["slots"], x["pos"],
            x["heldo"], x["counts"], x["mask"], None)

    for name in ("ctx", "new", "held", "table", "free", "start", "slots", "pos", "heldo",
                 "counts", "mask"):
        assert call(**{name: None}) == 1, name
        assert call(**{name: ok[name] + 2}) == 1, name
    assert call(R=-1) == 1 and call(pages=0) == 1 and call(T=-1) == 1 and call(nfree=-1) == 1
    assert call(P=0) == 1 and call(width=0) == 1 and call(par=None) == 1
    assert call(P=24) == 2 and call(P=8) == 2 and call(P=256) == 2 and call(R=16385) == 2
    assert call(pages=1 << 31) == 2 and call(T=1 << 31) == 2
    # outputs on inputs, or on each other
    assert call(heldo=a[2]) == 1 and call(slots=a[8]) == 1 and call(counts=a[0] + 4) == 1
    assert call(mask=a[3]) == 1


def test_write_refusals(lib):
    a = [_addr(i) for i in range(5)]

    def call(k=a[0], v=a[1], T=3, H=2, D=64, kt=128, kh=64, vt=128, vh=64, slots=a[2], kc=a[3],
             vc=a[4], pages=4, P=16):
        return lib.swiglu_cache_write(k, v, T, H, D, kt, kh, vt, vh, slots, kc, vc, pages, P, None)

    for bad in (dict(k=None), dict(v=None), dict(slots=None), dict(kc=None), dict(vc=None),
                dict(T=-1), dict(H=0), dict(pages=0), dict(k=a[0] + 8), dict(vc=a[4] + 2),
                dict(slots=a[2] + 1), dict(kt=129), dict(vh=-8), dict(kc=a[0]), dict(vc=a[3]),
                dict(vc=a[2]), dict(kt=1 << 31)):
        assert call(**bad) == 1, bad
    for bad in (dict(D=80), dict(P=48), dict(pages=1 << 28), dict(T=1 << 31), dict(H=65536)):
        assert call(**bad) == 2, bad


def test_attention_refusals(lib):
    a = [_addr(i) for i in range(9)]

    def call(q=a[0], qt=256, qh=64, k=a[1], v=a[2], pages=4, P=16, table=a[3], R=2, mp=4,
             ctx=a[4], start=a[5], mask=a[6], words=1, scale=0.125, out=a[7], T=3, Hq=4, Hkv=2,
             D=64, ws=a[8], nws=1 << 28):
        return lib.swiglu_tree_attention(q, qt, qh, k, v, pages, P, table, R, mp, ctx, start, mask,
                                         words, scale, out, T, Hq, Hkv, D, ws, nws, None)

    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(table=None), dict(ctx=None),
                dict(start=None), dict(out=None), dict(mask=None), dict(words=0), dict(words=-1),
                dict(T=-1), dict(R=-1), dict(Hq=3), dict(Hq=0), dict(mp=0), dict(q=a[0] + 8),
                dict(out=a[7] + 4), dict(mask=a[6] + 4), dict(ctx=a[4] + 1), dict(qt=250),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=0.0),
                dict(scale=-1.0), dict(out=a[0]),
                dict(out=a[1]), dict(out=a[2])):
        assert call(**bad) == 1, bad
    for bad in (dict(D=96), dict(P=20), dict(T=1 << 31), dict(mp=1 << 31), dict(words=1 << 21),
                dict(Hq=258)):
        assert call(**bad) == 2, bad


def test_accept_refusals(lib):
    a = [_addr(i) for i in range(7)]

    def call(k=a[0], v=a[1], L=2, pages=4, H=2, P=16, D=64, table=a[2], R=2, mp=4, ctx=a[3],
             paths=a[4], width=3, lens=a[5], out=a[6]):
        return lib.swiglu_cache_accept(k, v, L, pages, H, P, D, table, R, mp, ctx, paths, width,
                                       lens, out, None)

    for bad in (dict(k=None), dict(v=None), dict(table=None), dict(ctx=None), dict(paths=None),
                dict(lens=None), dict(out=None), dict(L=0), dict(R=-1), dict(mp=0),
                dict(width=-1), dict(k=a[0] + 8), dict(out=a[6] + 2), dict(v=a[0]),
                dict(out=a[3]), dict(out=a[0] + 64)):
        assert call(**bad) == 1, bad
    for bad in (dict(D=32), dict(P=12), dict(L=65536), dict(pages=1 << 28)):
        assert call(**bad) == 2, bad


def test_binding_refuses_host_tensors(lib):
    import torch
    import gemm_swiglu_mlp_gb300 as sg
    i = torch.zeros(2, dtype=torch.int32)
    c = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        sg.swiglu_cache_plan(i, i, i, torch.zeros(2, 2, dtype=torch.int32), i, 16, 4)
    with pytest.raises(TypeError):
        sg.swiglu_cache_write(c[:, :, 0], c[:, :, 0], i, c, c)
    with pytest.raises(TypeError):
        sg.swiglu_tree_attention(c[:, :, 0], c, c, i[:, None], i, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError):
        sg.swiglu_cache_accept(c, c, i[:, None], i, i[:, None], i)
