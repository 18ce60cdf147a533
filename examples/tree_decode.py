"""Decoding with trees of drafts: several samples of each prompt over shared pages, the tree's attention,
sampling at every node, and the accepted path.

A toy transformer with random weights (attention blocks only: an Engram layer's streaming state follows one
path, not a tree) continues prompts.  The samples of a prompt share its pages until they write into one.
Every step feeds, for each sequence, its last token and a tree of what followed earlier occurrences of its
final tokens; one pass gives the logits of all of them, a token is drawn after each, and the path that the
drawn tokens take down the tree is kept: its keys and values are moved together, the others' slots are
overwritten by the next step.

    python -m examples.tree_decode             # bf16, sampled
    python -m examples.tree_decode --greedy    # the same tokens with and without trees (fp32)
"""
from __future__ import annotations

import argparse
from dataclasses import dataclass
from typing import List, Tuple

import torch

from hashed_gram_embedding_engram_gb300 import (AttentionPlan, DraftTree, PagedCache, PagePool, SequenceBatch,
                                                sample_tokens)


@dataclass
class Shape:
    vocab: int = 64             # small, so that its n-grams recur
    d: int = 256
    heads: int = 4
    heads_kv: int = 2
    head_dim: int = 64
    page: int = 16
    layers: int = 2
    dtype: str = "bf16"


def rms_norm(x: torch.Tensor) -> torch.Tensor:
    y = x.float()
    return (y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


def int32(x) -> torch.Tensor:
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Model:
    """`rows` sequences of at most `longest` tokens, their pages in one pool."""

    def __init__(self, s: Shape, rows: int, longest: int):
        self.shape = s
        dt = torch.float32 if s.dtype == "f32" else torch.bfloat16
        g = torch.Generator(device="cuda").manual_seed(11)

        def normal(*size, std=1.0):
            return (torch.randn(size, generator=g, device="cuda") * std).to(dt)

        self.plan = AttentionPlan(heads=s.heads, heads_kv=s.heads_kv, head_dim=s.head_dim, page=s.page, dtype=s.dtype)
        per = -(-longest // s.page)
        self.pool = PagePool.empty(self.plan, rows, per, rows * (per + 1))
        self.caches = [PagedCache.empty(self.plan, rows * (per + 1)) for _ in range(s.layers)]
        self.rope = self.plan.rope_table(longest)
        self.ones = torch.ones(s.head_dim, device="cuda")
        self.qkv = [normal((s.heads + 2 * s.heads_kv) * s.head_dim, s.d, std=s.d ** -0.5) for _ in range(s.layers)]
        self.out = [normal(s.d, s.heads * s.head_dim, std=s.d ** -0.5) for _ in range(s.layers)]
        self.embed, self.head = normal(s.vocab, s.d), normal(s.vocab, s.d)

    def reserve(self, before: torch.Tensor, after: torch.Tensor) -> None:
        pairs, missing = self.pool.reserve(before, after)
        assert int(missing) == 0, int(missing)
        for cache in self.caches:
            cache.copy_pages(pairs)

    def forward(self, batch: SequenceBatch, tree: DraftTree, ids: torch.Tensor) -> torch.Tensor:
        """Logits [tokens, vocab] of a batch's new tokens."""
        s, T = self.shape, ids.shape[0]
        h = self.embed[ids.long()]
        for cache, w_qkv, w_out in zip(self.caches, self.qkv, self.out):
            q, k, v = (rms_norm(h) @ w_qkv.T).view(T, -1, s.head_dim).split((s.heads, s.heads_kv, s.heads_kv), 1)
            q, k = self.plan.qk_norm_rope(q, k, tree.positions, self.rope, g_q=self.ones, g_k=self.ones)
            cache.append(batch, k, v)
            attended, _ = cache.attend_tree(tree, q)
            h = h + attended.view(T, -1) @ w_out.T
        return (rms_norm(h) @ self.head.T).float() * (4 * s.d ** -0.5)


def draft_tree(text: List[int], branches: int, depth: int) -> Tuple[List[int], List[int]]:
    """(tokens, parents): the text's last token, and below it up to `depth` tokens of what followed each of
    the last `branches` earlier occurrences of its final two, common beginnings once."""
    tokens, parents, found = [text[-1]], [-1], 0
    for at in range(len(text) - 3, -1, -1):
        if found == branches:
            break
        if text[at:at + 2] != text[-2:]:
            continue
        found += 1
        node = 0
        for x in text[at + 2:at + 2 + depth]:
            child = next((i for i in range(node + 1, len(tokens)) if parents[i] == node and tokens[i] == x), None)
            if child is None:
                child = len(tokens)
                tokens.append(x)
                parents.append(node)
            node = child
    return tokens, parents


def generate(shape: Shape, prompts: List[List[int]], samples: int, new_tokens: int, branches: int, depth: int = 4,
             temperature: float = 0.0, top_p: float = 1.0, seed: int = 0):
    """`samples` continuations of each prompt by new_tokens tokens, with trees of up to `branches` lookups
    (0: none).  Returns the texts, the mean number of tokens a step, and the model."""
    P, B = len(prompts), len(prompts) * samples
    most = 1 + branches * depth
    model = Model(shape, P + B, max(map(len, prompts)) + new_tokens + most)
    g = torch.Generator(device="cuda").manual_seed(seed)
    pool = model.pool

    # the prompts but their last tokens, as chains; then the samples share their pages
    fed = [len(p) - 1 for p in prompts]
    model.reserve(int32([0] * (P + B)), int32(fed + [0] * B))
    start = [0]
    for n in fed:
        start.append(start[-1] + n)
    batch = SequenceBatch(int32(start), int32(fed), pool.table[:P], max_new=max(fed))
    chain = [i - 1 for n in fed for i in range(n)]
    model.forward(batch, DraftTree(model.plan, batch, int32(chain), max_nodes=max(fed)),
                  int32([x for p in prompts for x in p[:-1]]))
    rows = list(range(P, P + B))
    shared = [n for n in fed for _ in range(samples)]
    pool.fork(int32([p for p in range(P) for _ in range(samples)]), int32(rows), int32(shared))
    pool.free(int32(list(range(P))), int32([0] * P))

    text = [list(p) for p in prompts for _ in range(samples)]
    length, none = int32(shared), int32([0] * P)
    ends = [len(t) + new_tokens for t in text]
    steps = 0
    while any(len(t) < end for t, end in zip(text, ends)):
        # a sequence that has all its tokens feeds none
        trees = [draft_tree(t, branches, depth) if len(t) < end else ([], []) for t, end in zip(text, ends)]
        new = int32([len(t) for t, _ in trees])
        start = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
        start[1:] = new.cumsum(0)
        model.reserve(torch.cat((none, length)), torch.cat((none, length + new)))
        batch = SequenceBatch(start, length + new, pool.table[P:], max_new=most)
        tree = DraftTree(model.plan, batch, int32([p for _, parents in trees for p in parents]), max_nodes=most)
        ids = int32([x for tokens, _ in trees for x in tokens])
        logits = model.forward(batch, tree, ids)
        u = torch.rand(ids.shape[0], generator=g, device="cuda")
        sampled = sample_tokens(logits, u, temperature=temperature, top_p=top_p)
        path, count, emitted, length = tree.accept(ids, sampled, width=depth + 1)
        for cache in model.caches:
            cache.compact(batch, path, count)
        pool.free(int32(rows), length)             # pages that only dropped drafts had
        for t, n, out in zip(text, count.tolist(), emitted.tolist()):
            t += out[:n]
            steps += n > 0
    status, _ = model.plan.get_error()
    assert status == 0, status
    made = sum(len(t) for t in text) - sum(len(p) * samples for p in prompts)
    return text, made / max(steps, 1), model


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--greedy", action="store_true")
    p.add_argument("--prompts", type=int, default=3)
    p.add_argument("--samples", type=int, default=4)
    p.add_argument("--new-tokens", type=int, default=48)
    p.add_argument("--branches", type=int, default=3)
    a = p.parse_args()
    shape = Shape(dtype="f32" if a.greedy else "bf16")
    g = torch.Generator().manual_seed(1)
    prompts = torch.randint(0, shape.vocab, (a.prompts, 37), generator=g).tolist()
    how = dict(temperature=0.0) if a.greedy else dict(temperature=0.8, top_p=0.9)
    text, rate, _ = generate(shape, prompts, a.samples, a.new_tokens, a.branches, **how)
    print(f"{rate:.2f} tokens a step with trees of {a.branches} branches; first text continues {text[0][37:53]}")
    if a.greedy:
        plain, _, _ = generate(shape, prompts, a.samples, a.new_tokens, 0)
        n = min(len(x) for x in text + plain)
        print("the same tokens without trees:", all(x[:n] == y[:n] for x, y in zip(text, plain)))


if __name__ == "__main__":
    main()
