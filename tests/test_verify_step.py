"""The example decoder: its accepted paths (CPU), and on the GPU its caches and
choices against a dense forward pass of the whole sequences in 64 bits."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location(
    "verify_step", os.path.join(ROOT, "examples", "verify_step.py"))
ex = importlib.util.module_from_spec(spec)
spec.loader.exec_module(ex)


def test_accepted_paths():
    parents = torch.tensor([ex.TREE] * 4, dtype=torch.int32)
    tokens = torch.tensor([[9, 1, 2, 3, 4, 5, 6]] * 4)
    following = torch.tensor([[1, 3, 0, 5, 0, 7, 0],     # the whole first chain
                              [2, 3, 4, 5, 0, 0, 0],     # two of the second
                              [8, 3, 4, 5, 6, 0, 0],     # none: 1 and 2 do not follow 9
                              [1, 0, 4, 5, 6, 0, 0]])    # one; the second chain's do not hold
    paths, lens = ex.accepted(tokens, parents, following)
    assert lens.tolist() == [4, 3, 1, 2]
    assert [p[:n] for p, n in zip(paths.tolist(), lens.tolist())] == [
        [0, 1, 3, 5], [0, 2, 4], [0], [0, 1]]


def dense(weights, seq):
    """Logits [n, VOCAB], keys and values per layer [n, KV_HEADS, HEAD], in 64
    bits (weights as they are, nothing rounded)."""
    n = len(seq)
    x = weights["embed"].double()[torch.tensor(seq)]
    pos = torch.arange(n)
    caches = []

    def norm(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    for w in weights["layers"]:
        w = {k: v.double() for k, v in w.items()}
        h = (norm(x) @ w["qkv"]).view(n, -1, ex.HEAD)
        turned = ex.rotate(h[:, :ex.Q_HEADS + ex.KV_HEADS], pos)
        q, k = turned[:, :ex.Q_HEADS], turned[:, ex.Q_HEADS:]
        v = h[:, ex.Q_HEADS + ex.KV_HEADS:]
        caches.append((k, v))
        group = ex.Q_HEADS // ex.KV_HEADS
        s = torch.einsum("thd,xhd->htx", q, k.repeat_interleave(group, 1)) * ex.HEAD ** -0.5
        s = s.masked_fill(torch.ones(n, n).triu(1).bool(), float("-inf")).softmax(-1)
        x = x + torch.einsum("htx,xhd->thd", s, v.repeat_interleave(group, 1)).reshape(n, -1) @ w["o"]
        a = norm(x)
        x = x + (torch.nn.functional.silu(a @ w["w1"]) * (a @ w["w2"])) @ w["w3"]
    return norm(x) @ weights["head"].double(), caches


# What BF16 rounding explains: about ten roundings a layer (norm, qkv, rotation,
# weights, attention, o, norm, Y, out, two sums), each with 2^-9 / sqrt(3) =
# 1.1e-3 of root-mean-square relative error, in two layers and the head, none of
# which makes more than twice of it: sqrt(21) * 1.1e-3 * 2 = 1.0e-2. Twice that is
# allowed; a row out of place, a mask or position that is wrong gives about 1.
TOLERANCE = 2e-2


@pytest.mark.gpu
def test_generation_matches_a_dense_forward_pass():
    weights = ex.make_weights(2, seed=3)
    gen = torch.Generator().manual_seed(4)
    prompts = [torch.randint(ex.VOCAB, (n,), generator=gen).tolist() for n in (1, 17, 40)]
    steps = 12
    model = ex.Decoder(weights, 3, 40 + (steps + 1) * len(ex.TREE))
    seqs, gained = ex.generate(model, prompts, steps, seed=5)
    assert all(g >= 1 for g in gained)
    ctx, table = model.ctx.tolist(), model.table.cpu()
    for r, (prompt, seq) in enumerate(zip(prompts, seqs)):
        assert len(seq) == ctx[r] + 1   # the last token is not in the cache yet
        logits, caches = dense(weights, seq[:-1])
        # the chosen tokens are the largest, up to twice the logits' error
        chosen = logits[len(prompt) - 1:].gather(1, torch.tensor(seq[len(prompt):])[:, None])[:, 0]
        short = logits[len(prompt) - 1:].max(-1).values - chosen
        # (an error of one of 512 logits is within five of its deviations)
        assert short.max() <= 2 * 5 * TOLERANCE / 2 * logits.std()
        pages = table[r, torch.arange(ctx[r]) // ex.PAGE].long()
        rows = torch.arange(ctx[r]) % ex.PAGE
        for i, want in enumerate(caches):
            for cache, w in zip((model.k_cache, model.v_cache), want):
                got = cache[i].cpu()[pages, :, rows].double()
                err = (got - w).square().mean().sqrt() / w.square().mean().sqrt()
                assert err <= TOLERANCE, (r, i, err)


@pytest.mark.gpu
def test_drafts_do_not_change_what_is_cached():
    """Known sequences, drafted right in part: the caches' rows are those of the
    sequences, whichever branch of the tree they came by."""
    weights = ex.make_weights(2, seed=6)
    gen = torch.Generator().manual_seed(7)
    model = ex.Decoder(weights, 2, 96)
    prompts = [torch.randint(ex.VOCAB, (n,), generator=gen).tolist() for n in (15, 16)]
    last = model.prefill(prompts)
    seqs = [list(p) for p in prompts]
    parents = torch.tensor([ex.TREE] * 2, dtype=torch.int32, device="cuda")
    for step in range(4):
        drafts = torch.randint(ex.VOCAB, (2, len(ex.TREE)), generator=gen).cuda()
        drafts[:, 0] = last
        # find what follows, on the side by the first chain or the second
        first = 1 + step % 2
        for i in (first, first + 2, first + 4):
            lens = torch.full((2,), len(ex.TREE), dtype=torch.int32, device="cuda")
            following = model.forward(drafts.reshape(-1), lens, parents).argmax(-1).view(2, -1)
            drafts[:, i] = following[:, ex.TREE[i]]
        other = 3 - first
        drafts[:, other] = (drafts[:, first] + 1) % ex.VOCAB
        known = drafts.clone()
        following, lens, paths = model.verify(drafts, parents)
        for r in range(2):
            # (a tie within rounding may cut a path; what is accepted is cached)
            path = paths[r, :int(lens[r])].tolist()
            assert path == [0, first, first + 2, first + 4][:len(path)]
            seqs[r] += known[r, path].tolist()
        assert int(lens.min()) >= 2
        last = following.gather(1, (lens.long() - 1)[:, None])[:, 0]
    for r, seq in enumerate(seqs):
        n = int(model.ctx[r])
        assert n == len(seq)
        pages = model.table[r].cpu()[torch.arange(n) // ex.PAGE].long()
        rows = torch.arange(n) % ex.PAGE
        _, caches = dense(weights, seq)
        for i, want in enumerate(caches):
            for cache, w in zip((model.k_cache, model.v_cache), want):
                got = cache[i].cpu()[pages, :, rows].double()
                assert (got - w).square().mean().sqrt() <= TOLERANCE * w.square().mean().sqrt()
