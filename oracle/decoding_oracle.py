"""Restatement of the operators around the attention (the checker of the kernels): trees of drafted
tokens, pages shared among sequences, tokens from logits.

Plain Python and numpy, from the definitions in include/engram_attention.h; test infrastructure only.
"""
from __future__ import annotations

import math

import numpy as np

from oracle.attention_oracle import fix, fix_u, keys_of


# ---------------------------------------------------------------- trees
def layout(parent, start, length, window=0, most=256):
    """(sees: a bool matrix [n, n] for each sequence, positions [T]) of trees given by `parent` [T].  A row
    that does not see itself sees no key at all."""
    sees, positions = [], np.zeros(int(start[-1]), np.int64)
    for b in range(len(length)):
        n = int(start[b + 1] - start[b])
        see = np.zeros((n, n), bool)
        if n <= most and length[b] >= n:
            for i in range(n):
                line = [i]
                while 0 <= parent[start[b] + line[-1]] < line[-1]:
                    line.append(int(parent[start[b] + line[-1]]))
                if parent[start[b] + line[-1]] != -1:
                    continue
                see[i, line[:window] if window else line] = True
                positions[start[b] + i] = length[b] - n + len(line) - 1
        sees.append(see)
    return sees, positions


def tree_attention(q, k_pages, v_pages, start, length, table, scale, sees, positions, window=0):
    """q [T, H, D], pages [P, Hkv, page, D], all float64.  Returns out [T, H, D], lse [T, H] and mag
    [T, H, D] = sum softmax |v|."""
    T, H, D = q.shape
    page, Hkv = k_pages.shape[2], k_pages.shape[1]
    out, mag, lse = np.zeros((T, H, D)), np.zeros((T, H, D)), np.full((T, H), -np.inf)
    for b, m in enumerate(int(x) for x in length):
        n = int(start[b + 1] - start[b])
        if m < n:
            continue
        k, v = keys_of(k_pages, table[b], m, page), keys_of(v_pages, table[b], m, page)
        base = m - n
        for i in range(n):
            if not sees[b][i, i]:
                continue
            row = start[b] + i
            visible = np.zeros(m, bool)
            visible[max(0, max(positions[row], base) - window + 1) if window else 0:base] = True
            visible[base:] = sees[b][i]
            for h in range(H):
                g = h // (H // Hkv)
                s = scale * (k[visible, g] @ q[row, h])
                top = s.max()
                e = np.exp(s - top)
                lse[row, h] = top + math.log(e.sum())
                e /= e.sum()
                out[row, h] = e @ v[visible, g]
                mag[row, h] = e @ np.abs(v[visible, g])
    return out, lse, mag


def accept(parent, tokens, sampled, start, length, width):
    B = len(length)
    path, emitted = np.full((B, width), -1, np.int32), np.full((B, width), -1, np.int32)
    count, total = np.zeros(B, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        a, n = int(start[b]), int(start[b + 1] - start[b])
        at = 0 if n and length[b] >= n else None
        while at is not None and count[b] < width:
            path[b, count[b]], emitted[b, count[b]] = at, sampled[a + at]
            count[b] += 1
            at = next((i for i in range(at + 1, n) if parent[a + i] == at and tokens[a + i] == sampled[a + at]), None)
        total[b] = max(int(length[b]) - n, 0) + count[b]
    return path, count, emitted, total


# ---------------------------------------------------------------- pages
def compact(pages, table, start, length, path, count):
    """pages [P, heads, page, D] with the kept rows moved together."""
    out, page = pages.copy(), pages.shape[2]
    for b, c in enumerate(count):
        n = int(start[b + 1] - start[b])
        base = int(length[b]) - n
        row = [int(x) for x in path[b, :max(int(c), 0)]]
        if not 0 <= c <= path.shape[1] or base < 0 or any(not 0 <= x < n for x in row) or sorted(set(row)) != row:
            continue
        for i, x in enumerate(row):
            p, t = int(table[b][(base + x) // page]), int(table[b][(base + i) // page])
            if 0 <= p < len(pages) and 0 <= t < len(pages):
                out[t, :, (base + i) % page] = pages[p, :, (base + x) % page]
    return out


class Pool:
    def __init__(self, table, ref, page):
        self.table, self.ref, self.page = [list(map(int, r)) for r in table], [int(x) for x in ref], page

    def pages_of(self, tokens):
        return -(-int(tokens) // self.page)

    def free(self, rows, keep):
        for r, n in zip(rows, keep):
            if not 0 <= r < len(self.table) or n < 0:
                continue
            row = self.table[r]
            for g in range(self.pages_of(n), len(row)):
                if 0 <= row[g] < len(self.ref):
                    self.ref[row[g]] -= self.ref[row[g]] > 0
                    row[g] = -1

    def fork(self, src, dst, length):
        good = []
        for i, (a, d, n) in enumerate(zip(src, dst, length)):
            ok = 0 <= a < len(self.table) and 0 <= d < len(self.table) and 0 <= n <= len(self.table[0]) * self.page
            ok = ok and d not in src and list(dst).count(d) == 1
            ok = ok and all(e < 0 for e in self.table[d])
            ok = ok and all(0 <= e < len(self.ref) for e in self.table[a][:self.pages_of(n)])
            good.append(ok)
        for ok, a, d, n in zip(good, src, dst, length):
            for g in range(self.pages_of(n) if ok else 0):
                self.table[d][g] = self.table[a][g]
                self.ref[self.table[a][g]] += 1

    def reserve(self, before, after):
        """(pairs, missing)."""
        was, pairs = list(self.ref), [[-1, -1] for _ in self.table]
        unused = [i for i, x in enumerate(was) if x <= 0]
        wanted = []
        for r, (n0, n1) in enumerate(zip(before, after)):
            if n1 <= n0 or n0 < 0 or n1 > len(self.table[r]) * self.page:
                continue
            for g in range(n0 // self.page, self.pages_of(n1)):
                e = self.table[r][g]
                if e < 0 or (e < len(was) and was[e] > 1):
                    wanted.append((r, g))
        if len(wanted) > len(unused):
            return pairs, len(wanted) - len(unused)
        for (r, g), fresh in zip(wanted, unused):
            e = self.table[r][g]
            if e >= 0:
                self.ref[e] -= 1
                if g * self.page < before[r]:
                    pairs[r] = [e, fresh]
            self.table[r][g] = fresh
            self.ref[fresh] += 1
        return pairs, 0


# ---------------------------------------------------------------- sampling
_P = tuple(np.float32(x) for x in (1.0, -0.6931472, 0.24022648, -0.055503324, 0.009618437, -0.0013398875, 0.00015353362))


def weights(l, temperature):
    """The whole-number weights of a row of logits (float32, NaN as -inf): Python integers."""
    l = np.where(np.isnan(l), -np.inf, l).astype(np.float32)
    top = l.max()
    if top == -np.inf:
        return [0] * len(l)
    with np.errstate(all="ignore"):
        c = np.float32(1.4426950408889634) / np.float32(temperature)
        a = (top - l) * c
        a = np.where(np.isnan(a) | (a > 64), np.float32(64), a).astype(np.float32)
    a[l == top] = 0
    n = np.rint(a)
    f = a - n
    y = np.full_like(f, _P[6])
    for p in _P[5::-1]:
        y = y * f + p           # float32 arrays: each operation rounds
    assert y.dtype == np.float32
    return [0 if x == -np.inf else math.floor(math.ldexp(float(v), 38 - int(k))) for x, v, k in zip(l, y, n)]


def kept(l, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """({index: weight} of the tokens that a row keeps), greedy rows their one token."""
    l = np.where(np.isnan(l), -np.inf, np.asarray(l, np.float64))
    order = sorted(range(len(l)), key=lambda j: (-l[j], j))
    if l[order[0]] == -np.inf:
        return {}
    if not temperature > 0:
        return {order[0]: 1}
    w = weights(l, temperature)
    if 0 < top_k < len(l):
        order = order[:top_k]
    if top_p < 1:
        share = math.floor(max(float(np.float32(top_p)), 0.0) * 2 ** 24) * sum(w[j] for j in order)
        goal, run, n = max(1, -(-share // 2 ** 24)), 0, 0
        while n < len(order) and run < goal:
            run += w[order[n]]
            n += 1
        order = order[:n]
    return {j: w[j] for j in order if w[j] >= fix(np.float32(min_p))}


def sample(l, u, **settings):
    k = kept(l, **settings)
    total = sum(k.values())
    goal, run = fix_u(np.float32(u)) * total >> 24, 0
    for j in sorted(k):
        run += k[j]
        if run > goal:
            return j
    return -1
