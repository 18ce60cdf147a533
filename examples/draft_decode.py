"""Decoding with n-gram drafts: the Engram layer, the paged cache, attention and the draft check
in one loop.

A toy transformer with random weights (two blocks, each an Engram layer and an attention
sub-block) continues a prompt.  Every step feeds the last token and up to S drafted ones, taken
from the text so far (what followed the last occurrence of its final two tokens); the target's
probabilities of all of them come from one pass, and ``verify_drafts`` keeps a prefix of the
drafts and draws one more token.

What a rejected draft leaves behind: its keys and values lie past the sequence's length and are
overwritten by the next append; the Engram layer's streaming state is advanced by the kept tokens
only, from a copy taken before the step.

    python -m examples.draft_decode            # bf16, sampled
    python -m examples.draft_decode --greedy   # the same tokens with and without drafts (fp32)
"""
from __future__ import annotations

import argparse
from dataclasses import dataclass
from typing import List

import torch

import workloads as W
from hashed_gram_embedding_engram_gb300 import (AttentionPlan, EngramPlan, EngramState, EngramWeights, PagedCache,
                                                SequenceBatch, verify_drafts)


@dataclass
class Shape:
    vocab: int = 96             # small, so that its n-grams recur
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


class Layer:
    def __init__(self, shape: Shape, index: int, max_tokens: int, pages: int):
        w = W.TINY_F32.scaled(d=shape.d, row_dim=64, table_dtype="f32" if shape.dtype == "f32" else "bf16",
                              act_dtype=shape.dtype, V=shape.vocab)
        dt = torch.float32 if shape.dtype == "f32" else torch.bfloat16
        g = torch.Generator(device="cuda").manual_seed(100 + index)

        def normal(*size, std):
            return (torch.randn(size, generator=g, device="cuda") * std).to(dt)

        primes, mults = [1009, 1013, 1019, 1021], [2 * i + 3 for i in range(w.multiplier_count)]
        self.engram = EngramPlan(N=w.N, K=w.K, row_dim=64, d=shape.d, table_dtype=w.table_dtype, act_dtype=shape.dtype,
                                 primes=primes, multipliers=[m * 0x9E3779B97F4A7C15 % 2 ** 64 | 1 for m in mults],
                                 max_tokens=max_tokens)
        ones = torch.ones(shape.d, device="cuda")
        self.weights = EngramWeights(table=normal(sum(primes), 64, std=0.5),
                                     w_kv=normal(2 * shape.d, self.engram.d_mem, std=self.engram.d_mem ** -0.5),
                                     g_h=ones[None].contiguous(), g_k=ones[None].contiguous(), g_c=ones,
                                     conv=torch.full((shape.d, 4), 0.25, device="cuda"))
        self.attn = AttentionPlan(heads=shape.heads, heads_kv=shape.heads_kv, head_dim=shape.head_dim, page=shape.page,
                                  dtype=shape.dtype)
        self.cache = PagedCache.empty(self.attn, pages)
        self.g_q = torch.ones(shape.head_dim, device="cuda")
        self.g_k = torch.ones(shape.head_dim, device="cuda")
        rows = (shape.heads + 2 * shape.heads_kv) * shape.head_dim
        self.w_qkv = normal(rows, shape.d, std=shape.d ** -0.5)
        self.w_out = normal(shape.d, shape.heads * shape.head_dim, std=shape.d ** -0.5)
        self.state = None


class Model:
    """B sequences of at most `longest` tokens; `fed` counts the tokens in the caches."""

    def __init__(self, shape: Shape, B: int, longest: int, most_new: int):
        self.shape, self.B = shape, B
        per = -(-longest // shape.page)
        self.layers = [Layer(shape, i, B * most_new, B * per) for i in range(shape.layers)]
        for x in self.layers:
            x.state = EngramState.zeros(x.engram, B)
        # pages in an order of their own, as an allocator would hand them out
        g = torch.Generator().manual_seed(7)
        self.table = torch.randperm(B * per, generator=g).to(torch.int32).view(B, per).cuda()
        self.rope = self.layers[0].attn.rope_table(longest)
        dt = torch.float32 if shape.dtype == "f32" else torch.bfloat16
        g = torch.Generator(device="cuda").manual_seed(5)
        self.embed = torch.randn(shape.vocab, shape.d, generator=g, device="cuda").to(dt)
        self.head = torch.randn(shape.vocab, shape.d, generator=g, device="cuda").to(dt)
        self.proj = (torch.arange(shape.vocab, device="cuda", dtype=torch.int32) * 7 + 1) % 770
        self.fed = torch.zeros(B, dtype=torch.int32, device="cuda")

    def forward(self, ids: torch.Tensor) -> torch.Tensor:
        """Feed ids [B, T]; logits [B, T, V].  The Engram states are left as they were: the inputs
        are kept for `keep`."""
        s, (B, T) = self.shape, ids.shape
        start = torch.arange(0, B * T + 1, T, dtype=torch.int32, device="cuda")
        batch = SequenceBatch(start, self.fed + T, self.table, max_new=T)
        h = self.embed[ids.long()].contiguous()
        self._ids, self._inputs = ids, []
        for x in self.layers:
            self._inputs.append(h.clone())
            x.engram.forward(ids, self.proj, x.weights, h.view(B, T, 1, s.d), x.state.clone())
            qkv = (rms_norm(h) @ x.w_qkv.T).view(B * T, s.heads + 2 * s.heads_kv, s.head_dim)
            q, k, v = qkv.split((s.heads, s.heads_kv, s.heads_kv), 1)
            q = x.cache.append(batch, k, v, self.rope, g_k=x.g_k, q=q, g_q=x.g_q)
            out, _ = x.cache.attend(batch, q)
            h = h + (out.view(B, T, -1) @ x.w_out.T)
        return (rms_norm(h) @ self.head.T).float() * s.d ** -0.5

    def keep(self, count: List[int]) -> None:
        """The first count[b] of the tokens fed last stay; the others never were."""
        for x, h in zip(self.layers, self._inputs):
            for b, n in enumerate(count):
                if n:
                    x.engram.forward(self._ids[b:b + 1, :n].contiguous(), self.proj, x.weights,
                                     h[b:b + 1, :n].clone().view(1, n, 1, self.shape.d), x.state.rows(b, b + 1))
        self.fed += torch.tensor(count, dtype=torch.int32, device="cuda")


def draft(text: List[int], S: int) -> List[int]:
    """Up to S tokens that followed the last occurrence of the text's final two."""
    for at in range(len(text) - 3, -1, -1):
        if text[at:at + 2] == text[-2:]:
            return text[at + 2:at + 2 + S]
    return []


def generate(shape: Shape, prompts: torch.Tensor, new_tokens: int, S: int, greedy: bool, seed: int = 0):
    """Continue prompts [B, T] until one has new_tokens more, with up to S drafts a step (0: none).
    Returns the texts and the mean number of tokens a step."""
    B, T = prompts.shape
    model = Model(shape, B, T + new_tokens + S + 2, max(T, S + 1))
    text = prompts.tolist()
    g = torch.Generator(device="cuda").manual_seed(seed)

    def distribution(logits):
        if greedy:
            return torch.nn.functional.one_hot(logits.argmax(-1), shape.vocab).float()
        return torch.softmax(logits * 4, -1)

    def step(last, drafts, n_drafts):
        """Feed the last tokens and the drafts (none if S is 0); the check's answer."""
        p = distribution(model.forward(torch.cat((last, drafts), 1) if S else last))
        if not S:
            p = p.expand(B, 2, shape.vocab).contiguous()        # the row after no draft is not looked at
        u = torch.rand(B, drafts.shape[1] + 1, generator=g, device="cuda")
        return verify_drafts(p, drafts, u, n_drafts=n_drafts)     # lookups are certain: no draft probabilities

    # the prompt but its last token, which the first step feeds
    model.forward(prompts[:, :-1].to("cuda", torch.int32).contiguous())
    model.keep([T - 1] * B)
    steps = 0
    while max(len(t) for t in text) < T + new_tokens:
        width = max(S, 1)
        found = [draft(t, S) if S else [] for t in text]
        drafts = torch.tensor([f + [0] * (width - len(f)) for f in found], dtype=torch.int32, device="cuda")
        n = torch.tensor([len(f) for f in found], dtype=torch.int32, device="cuda")
        last = torch.tensor([[t[-1]] for t in text], dtype=torch.int32, device="cuda")
        tokens, accepted = step(last, drafts, n)
        a = accepted.tolist()
        for b, row in enumerate(tokens.tolist()):
            text[b] += row[:a[b] + 1]
        model.keep([x + 1 for x in a])
        steps += 1
    for x in model.layers:
        for status in (x.engram.get_error()[0], x.attn.get_error()[0]):
            assert status == 0, status
    made = sum(len(t) - T for t in text) / B
    return [t[:T + new_tokens] for t in text], made / max(steps, 1)


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--greedy", action="store_true")
    p.add_argument("--batch", type=int, default=4)
    p.add_argument("--new-tokens", type=int, default=64)
    p.add_argument("--drafts", type=int, default=4)
    a = p.parse_args()
    shape = Shape(dtype="f32" if a.greedy else "bf16")
    prompts = torch.randint(0, shape.vocab, (a.batch, 40), generator=torch.Generator().manual_seed(1))
    text, rate = generate(shape, prompts, a.new_tokens, a.drafts, a.greedy)
    print(f"{rate:.2f} tokens a step with {a.drafts} drafts; first text continues {text[0][40:56]}")
    if a.greedy:
        plain, _ = generate(shape, prompts, a.new_tokens, 0, True)
        n = min(len(x) for x in text + plain)
        print("the same tokens without drafts:", all(x[:n] == y[:n] for x, y in zip(text, plain)))


if __name__ == "__main__":
    main()
