"""Draws that fall among values which each count as 0 (below 2^-51), before the one that has
nearly all of the probability: some token with probability has to follow, never -1."""
import numpy as np
import pytest

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


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


# over one CTA a request and over several, with whole pieces and odd ones
@pytest.mark.parametrize("R,V", [(1, 31), (1, 1000), (1, 4096), (1, 32000), (2, 200003),
                                 (200, 33001), (160, 128000)])
@pytest.mark.parametrize("form", ["chain", "refused", "refused draft"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_draw_among_tiny_values(sg, R, V, form, dtype):
    n, refused = 2, V // 2
    target = torch.full((n * R, V), 2.0 ** -52, dtype=dtype, device="cuda")
    target[:, ::7] = 0                                # (tokens that cannot follow)
    target[:, V - 1] = 0.5
    target[:, refused] = 0.5
    tokens = np.full(n * R, refused if form != "chain" else -1)
    draft = None
    if form == "refused draft":
        draft = torch.zeros_like(target)
        draft[:, refused] = 1
    uniform = torch.zeros(n * R, device="cuda")
    uniform[1::2] = 0.75                              # (the drafted token does not hold)
    got = sg.swiglu_verify_drafts(i32(tokens), i32(np.arange(R + 1) * n), target, draft=draft,
                                  uniform=uniform, width=n)
    assert (got.path_lens == 1).all()
    nxt = got.next_tokens.long()
    assert (nxt >= 0).all(), nxt[nxt < 0].numel()
    assert (target[::2].gather(1, nxt[:, None]) > 0).all()
    if form != "chain":
        assert (nxt != refused).all()
    # a number inside the large value's share
    uniform[::2] = 0.99
    got = sg.swiglu_verify_drafts(i32(tokens), i32(np.arange(R + 1) * n), target, draft=draft,
                                  uniform=uniform, width=n)
    assert (got.next_tokens == V - 1).all()


def test_nothing_but_tiny_values(sg):
    # the pieces' sums count, no value does; and nothing counts at all: -1
    V = 64000
    target = torch.full((2, V), 2.0 ** -53, device="cuda")
    target[1] = 2.0 ** -80
    start, tokens = i32([0, 1, 2]), i32([0, 0])
    for u in (0.0, 0.3, 0.9999999):
        got = sg.swiglu_verify_drafts(tokens, start, target, width=1,
                                      uniform=torch.full((2,), u, device="cuda"))
        nxt = got.next_tokens.tolist()
        # (as exact as a piece, of 256 pieces: 16 CTAs of 16 warps)
        assert abs(nxt[0] / V - u) <= 1 / 256 + 1e-6 and nxt[1] == -1
