"""A small decoder that generates with drafted tokens over a paged cache, every
product of it by this library:

    python examples/verify_step.py [--requests 4] [--steps 24] [--layers 2]

Each step verifies a tree of drafted tokens per request: plan (pages, slots,
positions, masks), then per layer qkv product, cache write, tree attention and
gated MLP, then the accepted path is moved behind the context in all layers'
caches. Greedy: what comes out is what one token at a time would give, up to
ties within BF16 rounding. Weights are random; the sizes are the 0.5B MLP's (hidden 896,
intermediate 4864) with 14 query and 2 kv heads of 64. Norms, rotation and
drafting are plain PyTorch.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gemm_swiglu_mlp_gb300 as sg  # noqa: E402

HIDDEN, INNER, Q_HEADS, KV_HEADS, HEAD, VOCAB = 896, 4864, 14, 2, 64, 512
PAGE = 16
THETA = 10000.0


def make_weights(layers: int, seed: int = 0) -> dict:
    """Random BF16 weights, on the CPU."""
    gen = torch.Generator().manual_seed(seed)

    def mat(rows, cols):
        return (torch.randn(rows, cols, generator=gen) * rows ** -0.5).bfloat16()

    return {"embed": torch.randn(VOCAB, HIDDEN, generator=gen).bfloat16(),
            "head": mat(HIDDEN, VOCAB),
            "layers": [{"qkv": mat(HIDDEN, (Q_HEADS + 2 * KV_HEADS) * HEAD),
                        "o": mat(Q_HEADS * HEAD, HIDDEN),
                        "w1": mat(HIDDEN, INNER), "w2": mat(HIDDEN, INNER),
                        "w3": mat(INNER, HIDDEN)} for _ in range(layers)]}


def norm(x: torch.Tensor) -> torch.Tensor:
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


def rotate(x: torch.Tensor, positions: torch.Tensor) -> torch.Tensor:
    """x [tokens, heads, HEAD], halves rotated by position."""
    half = HEAD // 2
    freq = THETA ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
    angle = positions.double()[:, None, None] * freq
    a, b = x[..., :half].double(), x[..., half:].double()
    return torch.cat((a * angle.cos() - b * angle.sin(),
                      a * angle.sin() + b * angle.cos()), -1).to(x.dtype)


def accepted(tokens: torch.Tensor, parents: torch.Tensor, following: torch.Tensor):
    """Which drafts [R, n] hold: those whose parent does and is followed by
    them (siblings are different tokens, so they form one path from token 0).
    Returns paths [R, n] int32 (accepted indices first, increasing) and their
    lengths [R] int32."""
    R, n = tokens.shape
    holds = torch.zeros(R, n, dtype=torch.bool, device=tokens.device)
    holds[:, 0] = True
    for i in range(1, n):
        p = parents[:, i:i + 1].long()
        holds[:, i] = (holds.gather(1, p) & (following.gather(1, p) == tokens[:, i:i + 1]))[:, 0]
    paths = torch.sort((~holds).to(torch.uint8), dim=1, stable=True).indices
    return paths.int(), holds.sum(1).int()


class Decoder:
    def __init__(self, weights: dict, requests: int, max_context: int, device="cuda:0"):
        dev = torch.device(device)
        self.embed = weights["embed"].to(dev)
        self.head = sg.swiglu_pack_down_weights(weights["head"].to(dev))
        self.layers = [{"qkv": sg.swiglu_pack_down_weights(w["qkv"].to(dev)),
                        "o": sg.swiglu_pack_down_weights(w["o"].to(dev)),
                        "up": sg.swiglu_pack_weights(w["w1"].to(dev), w["w2"].to(dev)),
                        "down": sg.swiglu_pack_down_weights(w["w3"].to(dev))}
                       for w in weights["layers"]]
        per = (max_context + PAGE - 1) // PAGE
        pages = requests * per
        shape = (len(self.layers), pages, KV_HEADS, PAGE, HEAD)
        self.k_cache = torch.zeros(shape, dtype=torch.bfloat16, device=dev)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.table = torch.zeros(requests, per, dtype=torch.int32, device=dev)
        self.free = torch.randperm(pages, device=dev).int()   # any order will do
        self.free_head = torch.zeros(1, dtype=torch.int32, device=dev)
        self.held = torch.zeros(requests, dtype=torch.int32, device=dev)
        self.ctx = torch.zeros(requests, dtype=torch.int32, device=dev)

    def forward(self, tokens: torch.Tensor, new_lens: torch.Tensor, parents=None) -> torch.Tensor:
        """Logits [T, VOCAB] of the requests' new tokens, one after another in
        `tokens` [T]; their keys and values are in the caches afterwards, the
        context is as it was."""
        plan = sg.swiglu_cache_plan(self.ctx, new_lens, self.held, self.table, self.free, PAGE,
                                    tokens.numel(), parents=parents, free_head=self.free_head)
        self.held, self.free_head = plan.pages_held, plan.counts[2:3]
        q_end = Q_HEADS * HEAD
        x = self.embed[tokens.long()]
        for i, w in enumerate(self.layers):
            qkv = sg.swiglu_down_forward(norm(x), w["qkv"], q_end + 2 * KV_HEADS * HEAD)
            heads = qkv.view(-1, Q_HEADS + 2 * KV_HEADS, HEAD)
            turned = rotate(heads[:, :Q_HEADS + KV_HEADS], plan.positions)
            q, k, v = turned[:, :Q_HEADS], turned[:, Q_HEADS:], heads[:, Q_HEADS + KV_HEADS:]
            sg.swiglu_cache_write(k, v, plan.slots, self.k_cache[i], self.v_cache[i])
            att = sg.swiglu_tree_attention(q, self.k_cache[i], self.v_cache[i], self.table,
                                           self.ctx, plan.query_start, mask=plan.mask)
            x = x + sg.swiglu_down_forward(att.view(-1, q_end), w["o"], HIDDEN)
            x = x + sg.swiglu_mlp_forward(norm(x), w["up"], w["down"], INNER)
        return sg.swiglu_down_forward(norm(x), self.head, VOCAB)

    def prefill(self, prompts: list) -> torch.Tensor:
        """The prompts (lists of tokens) into the cache; returns the token that
        follows each."""
        dev = self.ctx.device
        lens = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device=dev)
        flat = torch.tensor([t for p in prompts for t in p], device=dev)
        logits = self.forward(flat, lens)
        self.ctx = self.ctx + lens
        return logits[lens.long().cumsum(0) - 1].argmax(-1)

    def verify(self, tokens: torch.Tensor, parents: torch.Tensor):
        """One step: trees of drafts [R, n] whose token 0 is the last known
        one. Returns (the token after each accepted one [R, n], how many were
        accepted [R], their indices [R, n]); the context grows by them."""
        R, n = tokens.shape
        new_lens = torch.full((R,), n, dtype=torch.int32, device=self.ctx.device)
        following = self.forward(tokens.reshape(-1), new_lens, parents).argmax(-1).view(R, n)
        paths, lens = accepted(tokens, parents, following)
        self.ctx = sg.swiglu_cache_accept(self.k_cache, self.v_cache, self.table, self.ctx, paths,
                                          lens)
        return following.gather(1, paths.long()), lens, paths


# A tree of 7: two chains of drafts from the last known token.
#   0 - 1 - 3 - 5
#     \ 2 - 4 - 6
TREE = (-1, 0, 0, 1, 2, 3, 4)


def generate(model: Decoder, prompts: list, steps: int, seed: int = 0):
    """Sequences (prompt and what follows) after `steps` verifications, and how
    many tokens each step gave. Drafts: what last followed the token, and a
    chain that starts from another token."""
    gen = torch.Generator().manual_seed(seed)
    R, dev = len(prompts), model.ctx.device
    last = model.prefill(prompts)
    seqs = [list(p) + [t] for p, t in zip(prompts, last.tolist())]
    successor = torch.randint(VOCAB, (R, VOCAB), generator=gen)
    parents = torch.tensor(TREE, dtype=torch.int32, device=dev).repeat(R, 1)
    gained = []
    for _ in range(steps):
        drafts = torch.zeros(R, len(TREE), dtype=torch.long)
        for r, s in enumerate(seqs):
            for a, b in zip(s[-9:-1], s[-8:]):
                successor[r, a] = b
            drafts[r, 0] = s[-1]
            for i, p in enumerate(TREE[1:], 1):
                drafts[r, i] = successor[r, drafts[r, p]]
            drafts[r, 2] = (drafts[r, 1] + 1 + torch.randint(VOCAB - 1, (1,), generator=gen)) % VOCAB
            for i in (4, 6):
                drafts[r, i] = successor[r, drafts[r, TREE[i]]]
        following, lens, _ = model.verify(drafts.to(dev), parents)
        for s, f, n in zip(seqs, following.tolist(), lens.tolist()):
            s.extend(f[:n])
        gained.append(lens.float().mean().item())
    sg.swiglu_check_device_status()
    return seqs, gained


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--steps", type=int, default=24)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--seed", type=int, default=0)
    args = ap.parse_args()
    gen = torch.Generator().manual_seed(args.seed)
    prompts = [torch.randint(VOCAB, (5 + 7 * r,), generator=gen).tolist()
               for r in range(args.requests)]
    longest = max(map(len, prompts)) + (args.steps + 1) * len(TREE)
    model = Decoder(make_weights(args.layers, args.seed), args.requests, longest)
    seqs, gained = generate(model, prompts, args.steps, args.seed)
    for p, s in zip(prompts, seqs):
        print("prompt of %d tokens, then %s" % (len(p), s[len(p):len(p) + 16]))
    print("%d steps, %.2f tokens a step and request" % (args.steps, sum(gained) / len(gained)))


if __name__ == "__main__":
    main()
