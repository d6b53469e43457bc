"""Greedy decoding with draft trees over the paged 8-bit cache.

A small random-weight transformer is the target model.  A prompt gets pages and
positions (kv_assign), its attention runs over its own keys (prompt_attention)
and the cache takes these in (kv_append).  Every step then drafts a tree of
tokens, runs all of its nodes through the target in one pass (kv_append, then
kv_attention with the tree's parents), verifies the logits (verify_tree) and
keeps the accepted path in the cache (kv_commit); pages of nodes that were
rejected go back.  The same tokens are then decoded one at a time, without
drafts, and compared.

    python examples/tree_decoding.py [--tokens N] [--batch B] [--seed S]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import draft_token_verification_sv_gb300 as sv

VOCAB, HIDDEN, LAYERS, HEADS, KV_HEADS, DIM, PAGE = 1000, 256, 2, 8, 2, 64, 16

# The tree: parent of every node, and which of its parent's best continuations it is.
PARENTS = (-1, 0, 0, 0, 1, 1, 2, 2, 3, 4, 4, 5, 6, 9, 9, 13)
CHOICE = (0, 0, 1, 2, 0, 1, 0, 1, 0, 0, 1, 0, 0, 0, 1, 0)
DEPTH = [0] * len(PARENTS)
for _i, _p in enumerate(PARENTS[1:], 1):
    DEPTH[_i] = DEPTH[_p] + 1


def norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


class Target:
    """The target model and its caches of `batch` sequences of up to `most` tokens."""

    def __init__(self, batch, most, seed, device):
        g = torch.Generator().manual_seed(seed)
        w = lambda *shape, gain=1.0: (torch.randn(*shape, generator=g) * gain / shape[0] ** 0.5).to(device)
        self.embed = torch.randn(VOCAB, HIDDEN, generator=g).to(device)
        self.unembed = w(HIDDEN, VOCAB)
        self.layers = [dict(qkv=w(HIDDEN, (HEADS + 2 * KV_HEADS) * DIM, gain=2.0), out=w(HEADS * DIM, HIDDEN, gain=0.3))
                       for _ in range(LAYERS)]
        pages = -(-most // PAGE)
        self.caches = [sv.kv_cache(batch * pages, KV_HEADS, DIM, PAGE, device) for _ in range(LAYERS)]
        self.pool = sv.kv_pool(batch * pages, device)
        self.table = torch.zeros(batch, pages, dtype=torch.int32, device=device)
        self.held = torch.zeros(batch, dtype=torch.int32, device=device)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.inv_freq = 10000.0 ** (-torch.arange(0, DIM, 2, device=device) / DIM)

    def score(self, tokens, parents=None, prompt=False):
        """Logits of new tokens [B, n] behind the cached ones, whose keys and values they join."""
        B, n = tokens.shape
        x = self.embed[tokens]
        position = sv.kv_assign(self.pool, self.table, self.held, self.lens, PAGE, max_new=n, parents=parents)["positions"]
        for w, cache in zip(self.layers, self.caches):
            q, k, v = (norm(x) @ w["qkv"]).view(B, n, -1, DIM).split((HEADS, KV_HEADS, KV_HEADS), 2)
            q, k = sv.rope(q, k, position, self.inv_freq, adjacent=True)
            sv.kv_append(cache, k, v, self.table, self.lens)
            seen = sv.prompt_attention(q, k, v) if prompt else sv.kv_attention(q, cache, self.table, self.lens, parents=parents)
            x = x + seen.flatten(2) @ w["out"]
        return norm(x) @ self.unembed

    def keep(self, lens):
        """The sequences' lengths from now on; pages that they no longer need go back."""
        self.lens = lens
        sv.kv_assign(self.pool, self.table, self.held, lens, PAGE)

    def draft(self, tokens):
        """The drafter: the target without its layers."""
        return sv.topk(norm(self.embed[tokens.long()]) @ self.unembed, max(CHOICE) + 1)


def prompt_of(batch, seed, device):
    return torch.randint(VOCAB, (batch, 37), generator=torch.Generator().manual_seed(seed + 1)).to(device)


def plain(batch, tokens, seed, device="cuda"):
    """Greedy decoding, one token a pass: [B, tokens]."""
    prompt = prompt_of(batch, seed, device)
    model = Target(batch, prompt.shape[1] + tokens + 1, seed, device)
    out = [model.score(prompt, prompt=True)[:, -1].argmax(-1)]
    model.lens += prompt.shape[1]
    while len(out) < tokens:
        out.append(model.score(out[-1][:, None])[:, -1].argmax(-1))
        model.lens += 1
    return torch.stack(out, 1)


def with_trees(batch, tokens, seed, device="cuda"):
    """The same with draft trees: [B, tokens] and the passes it took."""
    prompt = prompt_of(batch, seed, device)
    model = Target(batch, prompt.shape[1] + tokens + 2 * len(PARENTS), seed, device)
    root = model.score(prompt, prompt=True)[:, -1].argmax(-1)
    model.lens += prompt.shape[1]
    out = [[t] for t in root.tolist()]
    parents = torch.tensor(PARENTS, dtype=torch.int32, device=device).expand(batch, -1).contiguous()
    passes = 0
    while min(map(len, out)) < tokens:
        nodes = torch.zeros_like(parents)
        nodes[:, 0] = root
        for level in range(max(DEPTH)):
            for i in (i for i, d in enumerate(DEPTH) if d == level):
                best = model.draft(nodes[:, i])
                for child in (c for c, p in enumerate(PARENTS) if p == i):
                    nodes[:, child] = best[:, CHOICE[child]]
        got = sv.verify_tree(model.score(nodes, parents), parents, nodes, max(DEPTH))
        for cache in model.caches:
            new_lens = sv.kv_commit(cache, model.table, model.lens, got["path"], got["accept_len"], len(PARENTS))
        # a sequence that has its tokens stays where it is
        done = torch.tensor([len(o) >= tokens for o in out], device=device)
        model.keep(torch.where(done, model.lens, new_lens))
        kept, length = got["out_tokens"], got["accept_len"].long()
        root = torch.where(done, root, kept.gather(1, length[:, None])[:, 0].long())
        for o, row, n in zip(out, kept.tolist(), length.tolist()):
            if len(o) < tokens:
                o += row[:n + 1]
        passes += 1
    return torch.tensor([o[:tokens] for o in out], device=device), passes


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", type=int, default=64)
    p.add_argument("--batch", type=int, default=4)
    p.add_argument("--seed", type=int, default=0)
    args = p.parse_args()
    want = plain(args.batch, args.tokens, args.seed)
    got, passes = with_trees(args.batch, args.tokens, args.seed)
    print(f"{args.batch} sequences of {args.tokens} tokens: {args.tokens - 1} passes without drafts, {passes} with trees of {len(PARENTS)}")
    print("same tokens" if torch.equal(want, got) else f"{int((want != got).sum())} tokens differ")


if __name__ == "__main__":
    main()
