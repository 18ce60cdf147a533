"""float64 restatement of the attention sub-block's operators (the checker of the kernels).

Plain numpy loops over sequences and heads, from the definitions in
include/engram_attention.h; test infrastructure only.
"""
from __future__ import annotations

import math

import numpy as np


def norm_rope(x, g, eps, positions, rope, adjacent=False):
    """x [T, heads, D] float64; positions [T] (negative: not rotated); rope [length, r] or None."""
    y = np.array(x, np.float64)
    if g is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(g, np.float64)
    if rope is None or rope.shape[1] == 0:
        return y
    r = rope.shape[1]
    for t, p in enumerate(positions):
        if not 0 <= p < rope.shape[0]:
            continue
        c, s = rope[p, :r // 2].astype(np.float64), rope[p, r // 2:].astype(np.float64)
        lo = slice(0, r, 2) if adjacent else slice(0, r // 2)
        hi = slice(1, r, 2) if adjacent else slice(r // 2, r)
        a, b = y[t][:, lo].copy(), y[t][:, hi].copy()
        y[t][:, lo], y[t][:, hi] = a * c - b * s, a * s + b * c
    return y


def positions(start, length):
    """Position of each packed row; rows of no sequence get -1."""
    pos = np.full(int(start[-1]), -1, np.int64)
    for b in range(len(length)):
        n = start[b + 1] - start[b]
        pos[start[b]:start[b + 1]] = length[b] - n + np.arange(n)
    return pos


def keys_of(pages, table_row, length, page):
    """[length, heads, D] of one sequence."""
    if length == 0:
        return np.zeros((0, pages.shape[1], pages.shape[3]))
    return np.stack([pages[table_row[j // page], :, j % page] for j in range(length)])


def attention(q, k_pages, v_pages, start, length, table, scale, causal=True, window=0):
    """q [T, H, D], pages [P, Hkv, page, D], all float64.  Returns out [T, H, D], lse [T, H] and
    mag [T, H, D] = sum softmax |v| (what rounding errors scale with)."""
    T, H, D = q.shape
    page, Hkv = k_pages.shape[2], k_pages.shape[1]
    out, mag = np.zeros((T, H, D)), np.zeros((T, H, D))
    lse = np.full((T, H), -np.inf)
    for b in range(len(length)):
        n, m = start[b + 1] - start[b], int(length[b])
        k, v = keys_of(k_pages, table[b], m, page), keys_of(v_pages, table[b], m, page)
        for i in range(n):
            p = m - n + i
            if p < 0:
                continue
            hi = p + 1 if causal else m
            lo = max(0, p - window + 1) if window else 0
            if lo >= hi:
                continue
            for h in range(H):
                g = h // (H // Hkv)
                s = scale * (k[lo:hi, g] @ q[start[b] + i, h])
                top = s.max()
                e = np.exp(s - top)
                lse[start[b] + i, h] = top + math.log(e.sum())
                e /= e.sum()
                out[start[b] + i, h] = e @ v[lo:hi, g]
                mag[start[b] + i, h] = e @ np.abs(v[lo:hi, g])
    return out, lse, mag


def fix(x) -> int:
    """floor(x clamped to [0, 1] * 2^38), NaN: 0."""
    x = float(x)
    return 0 if not x > 0 else math.floor(min(x, 1.0) * 2 ** 38)


def fix_u(u) -> int:
    u = float(u)
    return 0 if not u > 0 else math.floor(min(u, 1.0 - 2.0 ** -24) * 2 ** 24)


def verify(target, draft, drafts, n_drafts, u):
    """Whole-number check of drafts, one sequence after another (draft may be None)."""
    B, S1, V = target.shape
    S = S1 - 1
    tokens, accepted = np.full((B, S1), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        n = S if n_drafts is None else min(max(int(n_drafts[b]), 0), S)
        a = 0
        while a < n:
            x = int(drafts[b, a])
            if not 0 <= x < V:
                break
            q = 2 ** 38 if draft is None else fix(draft[b, a, x])
            if not fix_u(u[b, a]) * q < fix(target[b, a, x]) * 2 ** 24:
                break
            tokens[b, a] = x
            a += 1
        w = [fix(x) for x in target[b, a]]
        if a < n:
            if draft is None:
                rest = [0 if j == int(drafts[b, a]) else x for j, x in enumerate(w)]
            else:
                rest = [max(x - fix(y), 0) for x, y in zip(w, draft[b, a])]
            w = rest if sum(rest) else w
        total = sum(w)
        goal, run = fix_u(u[b, S]) * total >> 24, 0
        for j, x in enumerate(w):
            run += x
            if run > goal:
                tokens[b, a] = j
                break
        accepted[b] = a
    return tokens, accepted
