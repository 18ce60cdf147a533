"""Cases and plain forms of the operators for decoding with trees of drafts over the paged cache.

tree      a tree of drafted tokens: its layout (who sees whom, positions) and its attention over the cache
sample    tokens from logits: temperature, top-k, top-p and min-p, from given random numbers
accept    the walk down the tree that the sampled tokens decide, and the kept tokens' rows moved together
compact   kept tokens of long sequences moved together, in place
pages     rows of the page table freed, forked and extended (copy on write), and the pages copied
"""
import math
import random

import numpy as np
import torch

own = False

# the layer widths this repository works with, as heads: d = 1024 (8 x 128 or 16 x 64), d = 4096 (32 x 128)
_HEADS = ((8, 2, 128), (16, 4, 64), (32, 8, 128))
_VOCAB = 129280
# 2^-f on [-1/2, 1/2], a weighted least-squares fit with P(0) = 1; relative error 1.0e-7 with the roundings
_EXP = (1.0, -0.6931472, 0.24022648, -0.055503324, 0.009618437, -0.0013398875, 0.00015353362)
_LOG2E = 1.4426950408889634


def listed():
    return [
        # one interactive sequence early in its answer with a small tree of drafts: latency
        dict(name="tree_one", op="tree", dtype="bf16", B=1, heads=8, heads_kv=2, head_dim=128, page=16, nodes_min=26,
             nodes_max=26, len_min=517, len_max=517, window=0, idle=0),
        # a serving batch at unequal lengths, trees of unequal size, an idle slot
        dict(name="tree_batch", op="tree", dtype="bf16", B=32, heads=32, heads_kv=8, head_dim=128, page=64, nodes_min=8,
             nodes_max=64, len_min=100, len_max=8192, window=0, idle=1),
        # few sequences with long contexts: the keys have to be split over the SMs
        dict(name="tree_long", op="tree", dtype="bf16", B=2, heads=16, heads_kv=4, head_dim=64, page=64, nodes_min=33,
             nodes_max=64, len_min=30011, len_max=65536, window=0, idle=0),
        # an fp32 layer with a sliding window
        dict(name="tree_window_f32", op="tree", dtype="f32", B=5, heads=16, heads_kv=4, head_dim=64, page=32, nodes_min=1,
             nodes_max=60, len_min=300, len_max=2500, window=512, idle=0),
        # one sequence's next token with the usual filters, one setting for all rows
        dict(name="sample_one", op="sample", dtype="f32", R=1, V=_VOCAB, mode="both", scalars=True),
        # the decode batch, each row with its request's own settings (greedy ones among them)
        dict(name="sample_batch", op="sample", dtype="f32", R=256, V=_VOCAB, mode="mixed", scalars=False),
        # the nodes of 16 trees, bf16 logits of a smaller vocabulary (many ties)
        dict(name="sample_nodes_bf16", op="sample", dtype="bf16", R=1024, V=32003, mode="topp", scalars=True),
        # the same interactive sequence's tree after sampling
        dict(name="accept_one", op="accept", dtype="bf16", B=1, heads_kv=2, head_dim=128, page=16, nodes_min=26,
             nodes_max=26, len_min=517, len_max=517),
        # the trees of a decode batch
        dict(name="accept_batch", op="accept", dtype="bf16", B=256, heads_kv=8, head_dim=128, page=64, nodes_min=1,
             nodes_max=64, len_min=64, len_max=2000),
        # half of four long prompts' tokens evicted
        dict(name="compact_long", op="compact", dtype="bf16", B=4, heads_kv=8, head_dim=128, page=64, len_min=9001,
             len_max=16384, sinks=4, keep=0.45),
        # a beam of four from one short prompt: latency
        dict(name="pages_beam", op="pages", dtype="bf16", prompts=1, children=4, heads_kv=2, head_dim=128, page=16,
             len_min=517, len_max=517, new=1),
        # sixteen samples of each of 32 prompts, their first tokens reserved
        dict(name="pages_fork", op="pages", dtype="bf16", prompts=32, children=16, heads_kv=8, head_dim=128, page=64,
             len_min=65, len_max=2049, new=40),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw(rng):
    op = rng.choice(("tree", "tree", "tree", "sample", "sample", "sample", "accept", "compact", "pages", "pages"))
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    if op == "sample":
        return dict(op=op, dtype=dtype, R=_log_int(rng, 1, 1024), V=rng.choice((_VOCAB, _log_int(rng, 1000, 200000))),
                    mode=rng.choice(("greedy", "temperature", "topk", "topp", "minp", "both", "mixed")),
                    scalars=rng.random() < 0.5)
    heads, heads_kv, head_dim = rng.choice(_HEADS)
    heads_kv = rng.choice([h for h in (1, heads_kv, heads_kv * 2, heads) if heads % h == 0 and heads // h <= 16])
    page = rng.choice((16, 32, 64, 128))
    shape = dict(heads_kv=heads_kv, head_dim=head_dim, page=page)
    if op == "tree":
        nodes = _log_int(rng, 1, 128 if dtype == "bf16" else 60)
        length = _log_int(rng, 16, 65536 if dtype == "bf16" else 2500)
        B = _log_int(rng, 1, 64)
        return dict(op=op, dtype=dtype, B=B, heads=heads, nodes_min=rng.randint(1, nodes), nodes_max=nodes,
                    len_min=rng.randint(0, length), len_max=length, window=rng.choice((0, 0, 0, _log_int(rng, 4, 4096))),
                    idle=rng.choice((0, 0, 1)) if B > 1 else 0, **shape)
    if op == "accept":
        nodes, length = _log_int(rng, 1, 128), _log_int(rng, 1, 4000)
        return dict(op=op, dtype=dtype, B=_log_int(rng, 1, 256), nodes_min=rng.randint(1, nodes), nodes_max=nodes,
                    len_min=rng.randint(0, length), len_max=length, **shape)
    if op == "compact":
        length = _log_int(rng, 200, 16384)
        return dict(op=op, dtype=dtype, B=_log_int(rng, 1, 16), len_min=rng.randint(100, length), len_max=length,
                    sinks=rng.randint(0, 8), keep=rng.choice((0.1, 0.25, 0.45)), **shape)
    length = _log_int(rng, 2, 4000)
    return dict(op=op, dtype=dtype, prompts=_log_int(rng, 1, 32), children=_log_int(rng, 1, 16),
                len_min=rng.randint(1, length), len_max=length, new=_log_int(rng, 1, 100), **shape)


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / (50 if case["dtype"] == "bf16" else 2))


def draw(rng):
    """A case of the listed ranges that costs no more than the largest listed one of its operator and type, whose
    cache and plain form stay under some 8 GB."""
    while True:
        case = _draw(rng)
        op = case["op"]
        limit = {"tree": 1.6e9, "sample": 1.4e8, "accept": 2e8, "compact": 2.5e8, "pages": 2e8}[op]
        padded = 1
        if op == "tree":
            L = case["len_max"] + case["nodes_max"]
            padded = case["B"] * L * max(case["heads"] * case["nodes_max"], case["heads_kv"] * case["head_dim"])
        elif op in ("accept", "compact"):
            padded = 2 * sum(_lengths(case)) * case["heads_kv"] * case["head_dim"]
        elif op == "pages":
            pages = sum(-(-m // case["page"]) for m in _lengths(case)) + case["prompts"] * case["children"] * 3
            padded = 2 * pages * case["page"] * case["heads_kv"] * case["head_dim"]
        if padded <= 2 ** 30 and _cost(case) <= limit:
            return case


# ---------------------------------------------------------------- what a case's sequences are
def _spread(lo, hi, n, salt):
    """n whole numbers over [lo, hi], both ends among them where n > 1, in an order of their own."""
    v = [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]
    random.Random(salt).shuffle(v)
    return v


def _lengths(case):
    """Cached tokens of each sequence (of each prompt)."""
    return _spread(case["len_min"], case["len_max"], case["prompts"] if case["op"] == "pages" else case["B"], 5)


def _nodes(case):
    return _spread(case["nodes_min"], case["nodes_max"], case["B"], 3)


def _idle(case):
    return {(b * 7 + 1) % case["B"] for b in range(case.get("idle", 0))}


def _tree(rng, n):
    """Parents of n nodes in the order of their depth (node 0 the text's last token), and a path down from node 0.
    The path's first draft comes after as many siblings as the path has nodes, as the likeliest one may."""
    if n < 8:
        return [-1] + list(range(n - 1)), list(range(rng.randint(1, n)))
    depth = rng.randint(2, min(6, n // 4 + 1))
    sizes = [depth + 1] + [1] * (depth - 1)
    for _ in range(n - 1 - sum(sizes)):
        sizes[rng.randrange(depth)] += 1
    parents, path, before = [-1], [0], [0]
    for size in sizes:
        level = list(range(len(parents), len(parents) + size))
        parents += [rng.choice(before) for _ in level]
        node = level[-1]
        parents[node] = path[-1]
        path.append(node)
        before = level
    return parents, path[:rng.randint(1, depth + 1)]


def _trees(case, seed):
    rng = random.Random(seed * 7919 + 11)
    return [_tree(rng, n) for n in _nodes(case)]


def _size(case):
    return 4 if case["dtype"] == "f32" else 2


def _torch_type(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def work(case):
    op, e = case["op"], _size(case)
    if op == "sample":
        # the logits; a weight (difference, product, polynomial, whole number) and its sums for each
        return dict(bytes=case["R"] * (case["V"] * e + 24), flops=18 * case["R"] * case["V"])
    row = case["heads_kv"] * case["head_dim"] * e
    if op == "tree":
        keys = pairs = 0
        w, idle, new, length = case["window"], _idle(case), _nodes(case), _lengths(case)
        for b, (n, m) in enumerate(zip(new, length)):
            if b in idle:
                continue
            seen = min(m, w - 1) if w else m
            keys += seen + n
            pairs += n * (seen + min(n, 5))     # a node has about five tokens of its tree behind it
        T = sum(new)
        return dict(bytes=2 * keys * row + T * case["heads"] * (2 * case["head_dim"] * e + 4) + 8 * T,
                    flops=4 * pairs * case["heads"] * case["head_dim"])
    if op == "accept":
        moved = sum(len(p) - 1 for (_, p), n in zip(_trees(case, 0), _nodes(case)) if n >= 8)
        return dict(bytes=4 * moved * row + 12 * sum(_nodes(case)) + 80 * case["B"], flops=0)
    if op == "compact":
        moved = sum(max(0, int(m * case["keep"]) - case["sinks"]) for m in _lengths(case))
        return dict(bytes=4 * moved * row + 4 * moved, flops=0)
    copied = sum(case["children"] for m in _lengths(case) if m % case["page"])
    entries = sum(-(-m // case["page"]) for m in _lengths(case)) * case["children"]
    return dict(bytes=4 * copied * case["page"] * row + 16 * entries, flops=0)


# ---------------------------------------------------------------- inputs
def _settings(case, g):
    """(temperature, top_k, top_p, min_p) of each row, or of all rows."""
    mode, R, V = case["mode"], case["R"], case["V"]
    if case["scalars"]:
        t, k, p, m = {"greedy": (0.0, 0, 1.0, 0.0), "temperature": (0.7, 0, 1.0, 0.0), "topk": (1.0, 40, 1.0, 0.0),
                      "topp": (0.9, 0, 0.92, 0.0), "minp": (1.2, 0, 1.0, 0.05), "both": (0.8, 50, 0.95, 0.0),
                      "mixed": (0.6, 200, 0.9, 0.01)}[mode]
        return t, k, p, m

    def uniform(lo, hi):
        return lo + (hi - lo) * torch.rand(R, generator=g, device="cuda")

    t, p, m = uniform(0.4, 1.5), uniform(0.5, 0.99), uniform(0.0, 0.1)
    k = torch.exp(uniform(0.0, math.log(min(V, 2000)))).to(torch.int32)
    use = {"greedy": (0, 0, 0, 0), "temperature": (1, 0, 0, 0), "topk": (1, 1, 0, 0), "topp": (1, 0, 1, 0),
           "minp": (1, 0, 0, 1), "both": (1, 1, 1, 0)}.get(mode)
    if use is None:
        # rows greedy, unfiltered, and with each filter and all of them
        kind = torch.arange(R, device="cuda") % 8
        use = (kind != 0, (kind == 2) | (kind >= 5), (kind == 3) | (kind == 5) | (kind == 7), (kind == 4) | (kind >= 6))
    else:
        use = [torch.full((R,), bool(x), device="cuda") for x in use]
    return (torch.where(use[0], t, 0.0), torch.where(use[1], k, 0).to(torch.int32), torch.where(use[2], p, 1.0),
            torch.where(use[3], m, 0.0))


def _table(g, used, per, spare):
    """A page table of rows that use so many pages, in an order of their own, over all pages and `spare` more."""
    pages = sum(used) + spare
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(used), per), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, m in enumerate(used):
        table[b, :m] = order[at:at + m]
        at += m
    return table, pages


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 29)
    dt, op = _torch_type(case), case["op"]

    def normal(*shape):
        out = torch.empty(shape, dtype=dt, device="cuda")
        return out.normal_(generator=g)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    if op == "sample":
        R, V = case["R"], case["V"]
        logits = torch.randn((R, V), generator=g, device="cuda").mul_(3.0)
        # a handful of likely tokens a row, and a tenth of the rows held to a grammar
        top = torch.randint(0, V, (R, 12), generator=g, device="cuda")
        logits.scatter_add_(1, top, 4 + 4 * torch.rand((R, 12), generator=g, device="cuda"))
        masked = torch.rand((R, 1), generator=g, device="cuda") < 0.1
        hidden = torch.rand((R, V), generator=g, device="cuda") < 0.98
        logits.masked_fill_(masked & hidden, -math.inf)
        t, k, p, m = _settings(case, g)
        return dict(logits=logits.to(dt), u=torch.rand((R,), generator=g, device="cuda"), temperature=t, top_k=k,
                    top_p=p, min_p=m)
    page, Hkv, D = case["page"], case["heads_kv"], case["head_dim"]
    length = _lengths(case)
    if op in ("tree", "accept"):
        new, idle = _nodes(case), _idle(case)
        trees = _trees(case, seed)
        total = [0 if b in idle else n + m for b, (n, m) in enumerate(zip(new, length))]
        used = [-(-m // page) for m in total]
        table, pages = _table(g, used, max(1, max(used)), 1)
        start = np.concatenate(([0], np.cumsum(new)))
        s = dict(start=ints(start.tolist()), length=ints(total), table=table,
                 parent=ints([p for parents, _ in trees for p in parents]), k_pages=normal(pages, Hkv, page, D),
                 v_pages=normal(pages, Hkv, page, D))
        if op == "tree":
            s["q"] = normal(int(start[-1]), case["heads"], D)
            return s
        token = np.random.RandomState(seed % 2 ** 31).randint(0, _VOCAB, int(start[-1]))
        sampled = np.random.RandomState((seed + 1) % 2 ** 31).randint(0, _VOCAB, int(start[-1]))
        for at, (_, path) in zip(start, trees):
            for x, y in zip(path, path[1:]):
                sampled[at + x] = token[at + y]
        s.update(token=ints(token.tolist()), sampled=ints(sampled.tolist()))
        return s
    if op == "compact":
        used = [-(-m // page) for m in length]
        table, pages = _table(g, used, max(used), 1)
        count = [min(m, max(case["sinks"], int(m * case["keep"]))) for m in length]
        path = torch.full((case["B"], max(count)), -1, dtype=torch.int32, device="cuda")
        for b, (m, c) in enumerate(zip(length, count)):
            # the first tokens, and the best of the later ones by some score
            sinks = min(c, case["sinks"])
            kept = torch.randperm(m - c, generator=g, device="cuda")[:c - sinks].sort().values + c
            path[b, :c] = torch.cat((torch.arange(sinks, device="cuda"), kept)).to(torch.int32)
        return dict(start=ints(np.concatenate(([0], np.cumsum(length))).tolist()), length=ints(length), table=table,
                    path=path, count=ints(count), k_pages=normal(pages, Hkv, page, D),
                    v_pages=normal(pages, Hkv, page, D))
    # rows: the prompts, then each prompt's children, which hold a few pages of the sequences they served before
    P, C, new = case["prompts"], case["children"], case["new"]
    used = [-(-m // page) for m in length] + [i % 3 for i in range(P * C)]
    per = max(max(-(-(m + new) // page) for m in length), 2)
    spare = P * C * (-(-new // page) + 1)
    table, pages = _table(g, used, per, spare)
    ref = torch.zeros(pages, dtype=torch.int32, device="cuda")
    ref[table[table >= 0].long()] = 1
    child = [m for m in length for _ in range(C)]
    return dict(table=table, ref=ref, rows=ints(list(range(P, P + P * C))), keep=ints([0] * (P * C)),
                src=ints([p for p in range(P) for _ in range(C)]), fork_length=ints(child), before=ints(length + child),
                after=ints(length + [m + new for m in child]), k_pages=normal(pages, Hkv, page, D),
                v_pages=normal(pages, Hkv, page, D))


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    op = case["op"]
    if own:
        import hashed_gram_embedding_engram_gb300 as E
        s["E"] = E
        if op == "sample":
            s["tokens"] = torch.empty((case["R"],), dtype=torch.int32, device="cuda")
            return s
        heads = case.get("heads", case["heads_kv"])
        s["plan"] = E.AttentionPlan(heads=heads, heads_kv=case["heads_kv"], head_dim=case["head_dim"], page=case["page"],
                                    dtype=case["dtype"])
        s["cache"] = E.PagedCache(s["plan"], s["k_pages"], s["v_pages"])
        if op == "pages":
            s["pool"] = E.PagePool(s["plan"], s["table"], s["ref"])
        else:
            s["batch"] = E.SequenceBatch(s["start"], s["length"], s["table"], max_new=case.get("nodes_max", 0))
        if op == "tree":
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
        if op == "accept":
            s["tree"] = E.DraftTree(s["plan"], s["batch"], s["parent"], max_nodes=case["nodes_max"])
    return s


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"tree": _plain_tree, "sample": _plain_sample, "accept": _plain_accept, "compact": _plain_compact,
                "pages": _plain_pages}[op](s)
    if op == "tree":
        tree = s["E"].DraftTree(s["plan"], s["batch"], s["parent"], max_nodes=s["case"]["nodes_max"],
                                window=s["case"]["window"])
        out, lse = s["cache"].attend_tree(tree, s["q"], out=s["out"], lse=s["lse"])
        return out, lse, tree.positions
    if op == "sample":
        return s["E"].sample_tokens(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                                    min_p=s["min_p"], tokens=s["tokens"])
    if op == "accept":
        path, count, tokens, length = s["tree"].accept(s["token"], s["sampled"], width=8)
        s["cache"].compact(s["batch"], path, count)
        return path, count, tokens, length, s["k_pages"], s["v_pages"]
    if op == "compact":
        s["cache"].compact(s["batch"], s["path"], s["count"])
        return s["k_pages"], s["v_pages"]
    s["pool"].free(s["rows"], s["keep"])
    s["pool"].fork(s["src"], s["rows"], s["fork_length"])
    pairs, missing = s["pool"].reserve(s["before"], s["after"])
    s["cache"].copy_pages(pairs)
    return pairs, missing, s["table"], s["ref"], s["k_pages"], s["v_pages"]


# ---------------------------------------------------------------- plain forms
def _plain_ancestors(s):
    """(rows [B, N] of the packed arrays, live [B, N], the nodes that each node sees [B, N, N])."""
    N, B = s["case"]["nodes_max"], s["case"]["B"]
    start, length = s["start"].long(), s["length"].long()
    new = start[1:] - start[:-1]
    i = torch.arange(N, device="cuda")
    rows = (start[:-1, None] + i).clamp(max=s["parent"].shape[0] - 1)
    live = (i < new[:, None]) & (length >= new)[:, None]
    parent = s["parent"].long()[rows]
    see = ((parent[:, :, None] == i) | torch.eye(N, dtype=torch.bool, device="cuda")) & live[:, :, None]
    see = see.float()
    reach = 1
    while reach < N:
        see = (torch.matmul(see, see) > 0).float()
        reach *= 2
    return rows, live, (see > 0) & live[:, None, :]


def _plain_tree(s):
    case, q = s["case"], s["q"]
    H, Hkv, D, page = case["heads"], case["heads_kv"], case["head_dim"], case["page"]
    B, N, L, w = case["B"], case["nodes_max"], s["table"].shape[1] * case["page"], case["window"]
    rows, live, see = _plain_ancestors(s)
    start, length = s["start"].long(), s["length"].long()
    new = start[1:] - start[:-1]
    base = (length - new).clamp(min=0)
    depth = (see.sum(2) - 1).clamp(min=0)
    at = torch.where(live, base[:, None] + depth, torch.zeros_like(depth))
    if w:
        see = see & (depth[:, None, :] > depth[:, :, None] - w)
    i, j = torch.arange(N, device="cuda"), torch.arange(L, device="cuda")
    seen = torch.zeros((B, N, L + 1), dtype=torch.bool, device="cuda")
    slot = torch.where(i < new[:, None], base[:, None] + i, torch.full_like(rows, L)).clamp(max=L)
    seen.scatter_(2, slot[:, None, :].expand(B, N, N), see)
    seen = seen[:, :, :L]
    cached = j < base[:, None, None]
    if w:
        cached = cached & (j > at[:, :, None] - w)
    seen = (seen | cached) & live[:, :, None]
    x = q[rows].float().view(B, N, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    table = s["table"].long().clamp(min=0)
    k = s["k_pages"][table].transpose(1, 2).reshape(B, Hkv, L, D).float()
    score = torch.matmul(x, k.transpose(2, 3)).mul_(1 / math.sqrt(D)).view(B, Hkv, H // Hkv, N, L)
    del k
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = score.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    v = s["v_pages"][table].transpose(1, 2).reshape(B, Hkv, L, D).float()
    out = torch.matmul(e.view(B, Hkv, -1, L), v).view(B, Hkv, H // Hkv, N, D)
    out = out / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + total.log()).squeeze(-1)
    row = torch.arange(q.shape[0], device="cuda")
    b = torch.searchsorted(start, row, right=True) - 1
    n = row - start[b]
    out = out.permute(0, 3, 1, 2, 4).reshape(B, N, H, D)[b, n]
    return out.to(q.dtype), lse.permute(0, 3, 1, 2).reshape(B, N, H)[b, n], at[b, n].to(torch.int32)


def _whole(x, bits):
    return (torch.nan_to_num(x.float(), nan=0.0).clamp(0, 1) * 2.0 ** bits).to(torch.int64)


def _plain_weights(l, temperature):
    """Whole numbers floor(2^38 E(a)), a = (max - l) log2(e) / temperature, in float operations that each round."""
    top = l.amax(1, keepdim=True)
    c = torch.full_like(temperature, _LOG2E) / temperature
    a = (top - l) * c[:, None]
    a = torch.where(l == -math.inf, torch.full_like(a, 64.0), a)
    a = torch.where(temperature[:, None] > 0, a, torch.full_like(a, 64.0))
    a = torch.where(l == top, torch.zeros_like(a), torch.nan_to_num(a, nan=64.0).clamp(max=64.0))
    n = torch.round(a)
    f = a - n
    y = torch.full_like(f, _EXP[6])
    y = y.mul_(f).add_(_EXP[5]).mul_(f).add_(_EXP[4]).mul_(f).add_(_EXP[3]).mul_(f).add_(_EXP[2])
    y = y.mul_(f).add_(_EXP[1]).mul_(f).add_(_EXP[0])
    y = (y.view(torch.int32) - (n.to(torch.int32) << 23)).view(torch.float32)
    w = (y.clamp(max=1.0) * 2.0 ** 38).to(torch.int64)
    return torch.where(top == -math.inf, torch.zeros_like(w), w)


def _share(part, total, up):
    """floor (or ceiling) of part * total / 2^24, with part < 2^24 and total < 2^62."""
    low = part * (total & (2 ** 24 - 1))
    return part * (total >> 24) + (low >> 24) + (((low & (2 ** 24 - 1)) > 0).long() if up else 0)


def _plain_sample(s):
    logits = s["logits"]
    R, V = logits.shape

    def row(x, dtype):
        return x.to(dtype) if isinstance(x, torch.Tensor) else torch.full((R,), x, dtype=dtype, device="cuda")

    temperature, top_p, min_p = (row(s[k], torch.float32) for k in ("temperature", "top_p", "min_p"))
    top_k = row(s["top_k"], torch.int64)
    l = torch.nan_to_num(logits.float(), nan=-math.inf, posinf=math.inf, neginf=-math.inf) + 0.0
    w = _plain_weights(l, temperature)
    order = torch.sort(l, dim=1, descending=True, stable=True).indices
    ranked = w.gather(1, order)
    k = torch.where((top_k <= 0) | (top_k > V), torch.full_like(top_k, V), top_k)
    ranked = torch.where(torch.arange(V, device="cuda") < k[:, None], ranked, torch.zeros_like(ranked))
    upto = ranked.cumsum(1)
    goal = _share(_whole(top_p.clamp(max=1.0), 24).clamp(max=2 ** 24 - 1), upto[:, -1], True).clamp(min=1)
    inside = (upto - ranked < goal[:, None]) | (top_p >= 1)[:, None]
    ranked = torch.where(inside & (ranked >= _whole(min_p, 38)[:, None]), ranked, torch.zeros_like(ranked))
    w = torch.zeros_like(w).scatter_(1, order, ranked)
    upto = w.cumsum(1)
    total = upto[:, -1]
    goal = _share((s["u"].clamp(0, 1 - 2.0 ** -24) * 2.0 ** 24).to(torch.int64), total, False)
    token = torch.where(temperature > 0, (upto <= goal[:, None]).sum(1), order[:, 0])
    return torch.where(total > 0, token, torch.full_like(token, -1)).to(torch.int32)


def _plain_move(s, path, count):
    """Rows base + path[b, i] of the cache to base + i, for i < count[b]."""
    page, start, length = s["case"]["page"], s["start"].long(), s["length"].long()
    base = length - (start[1:] - start[:-1])
    i = torch.arange(path.shape[1], device="cuda")
    b, i = torch.nonzero(i < count[:, None], as_tuple=True)
    source, to = base[b] + path.long()[b, i], base[b] + i
    table = s["table"].long()
    p, t = table[b, source // page], table[b, to // page]
    for pages in (s["k_pages"], s["v_pages"]):
        pages[t, :, to % page] = pages[p, :, source % page]


def _plain_accept(s):
    rows, live, see = _plain_ancestors(s)
    B, N = rows.shape
    W = 8
    token, sampled = s["token"].long()[rows], s["sampled"].long()[rows]
    parent = s["parent"].long()[rows]
    i = torch.arange(N, device="cuda")
    fits = (token == sampled.gather(1, parent.clamp(min=0))) & (parent >= 0) & live
    # of the children of one node that fit, the first
    same = (parent[:, :, None] == parent[:, None, :]) & fits[:, None, :] & (i[None, :] < i[:, None])
    good = (fits & ~same.any(2)) | (i == 0)
    kept = live & ~(see & ~good[:, None, :]).any(2)
    kept = kept & (see[:, :, 0])
    where = kept.long().cumsum(1) - 1
    path = torch.full((B, N + W + 1), -1, dtype=torch.int64, device="cuda")
    path.scatter_(1, torch.where(kept, where, torch.full_like(where, N + W)), i.expand(B, N).contiguous())
    path = path[:, :W].contiguous()
    count = kept.sum(1).clamp(max=W)
    out = torch.where(path >= 0, sampled.gather(1, path.clamp(min=0)), torch.full_like(path, -1))
    new = s["start"].long()[1:] - s["start"].long()[:-1]
    length = (s["length"].long() - new).clamp(min=0) + count
    _plain_move(s, path, count)
    i32 = torch.int32
    return path.to(i32), count.to(i32), out.to(i32), length.to(i32), s["k_pages"], s["v_pages"]


def _plain_compact(s):
    _plain_move(s, s["path"], s["count"].long())
    return s["k_pages"], s["v_pages"]


def _plain_pages(s):
    page, table, ref = s["case"]["page"], s["table"], s["ref"]
    S, P = table.shape
    g = torch.arange(P, device="cuda")
    # free the rows from the page after those that are kept
    rows = s["rows"].long()
    entry = table[rows]
    drop = (g >= ((s["keep"].long() + page - 1) // page)[:, None]) & (entry >= 0)
    ref.scatter_add_(0, entry.long().clamp(min=0).flatten(), -drop.flatten().to(torch.int32))
    table[rows] = torch.where(drop, torch.full_like(entry, -1), entry)
    # fork: the first pages of another row, shared
    used = (s["fork_length"].long() + page - 1) // page
    entry = torch.where(g < used[:, None], table[s["src"].long()], -1).to(torch.int32)
    ref.scatter_add_(0, entry.long().clamp(min=0).flatten(), (entry >= 0).flatten().to(torch.int32))
    table[rows] = entry
    # reserve: pages to be written get one of their own
    before, after = s["before"].long()[:, None], s["after"].long()[:, None]
    written = (g >= before // page) & (g < (after + page - 1) // page) & (after > before)
    shared = written & (table >= 0) & (ref[table.long().clamp(min=0)] > 1)
    need = (written & (table < 0)) | shared
    wanted = need.sum()
    unused = torch.sort((ref > 0).to(torch.int32), stable=True).indices
    missing = (wanted - (ref == 0).sum()).clamp(min=0)
    need, shared = need & (missing == 0), shared & (missing == 0)
    rank = (need.flatten().long().cumsum(0) - 1).clamp(min=0, max=unused.numel() - 1).view(S, P)
    fresh = unused[rank].to(torch.int32)
    copied = shared & (g * page < before)
    pairs = torch.full((S, 2), -1, dtype=torch.int32, device="cuda")
    any_copy, which = copied.any(1), copied.long().argmax(1, keepdim=True)
    pairs[:, 0] = torch.where(any_copy, table.gather(1, which)[:, 0], -1)
    pairs[:, 1] = torch.where(any_copy, fresh.gather(1, which)[:, 0], -1)
    ref.scatter_add_(0, table.long().clamp(min=0).flatten(), -shared.flatten().to(torch.int32))
    ref.scatter_add_(0, fresh.long().flatten(), need.flatten().to(torch.int32))
    table.copy_(torch.where(need, fresh, table))
    b = torch.nonzero(any_copy)[:, 0]
    for pages in (s["k_pages"], s["v_pages"]):
        pages[pairs[b, 1].long()] = pages[pairs[b, 0].long()]
    return pairs, missing.to(torch.int32)[None], table, ref, s["k_pages"], s["v_pages"]


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s, op = _inputs(case, seed), case["op"]
    if op == "sample":
        return _exact_sample(s)
    if op == "pages":
        return _exact_pages(case, s)
    if op == "tree":
        return _exact_tree(case, s)
    start, length = s["start"].tolist(), s["length"].tolist()
    k, v, B = s["k_pages"].double(), s["v_pages"].double(), case["B"]
    if op == "compact":
        _exact_move(case, s, (k, v), s["path"].tolist(), s["count"].tolist())
        return k, v
    token, sampled, parent = s["token"].tolist(), s["sampled"].tolist(), s["parent"].tolist()
    path, out = [[-1] * 8 for _ in range(B)], [[-1] * 8 for _ in range(B)]
    count = [0] * B
    for b in range(B):
        a, n = start[b], start[b + 1] - start[b]
        at = 0
        while at is not None and count[b] < 8 and n:
            path[b][count[b]], out[b][count[b]] = at, sampled[a + at]
            count[b] += 1
            at = next((i for i in range(at + 1, n) if parent[a + i] == at and token[a + i] == sampled[a + at]), None)
    _exact_move(case, s, (k, v), path, count)
    total = [m - (start[b + 1] - start[b]) + count[b] for b, m in enumerate(length)]
    return tuple(torch.tensor(x, dtype=torch.int32, device="cuda") for x in (path, count, out, total)) + (k, v)


def _exact_move(case, s, both, path, count):
    page, start, length = case["page"], s["start"].tolist(), s["length"].tolist()
    table = s["table"].tolist()
    for b, c in enumerate(count):
        base = length[b] - (start[b + 1] - start[b])
        a = [base + path[b][i] for i in range(c)]
        source = torch.tensor([table[b][x // page] * page + x % page for x in a], dtype=torch.int64, device="cuda")
        to = torch.tensor([table[b][x // page] * page + x % page for x in range(base, base + c)], dtype=torch.int64,
                          device="cuda")
        for pages in both:
            rows = pages.transpose(1, 2)
            moved = rows[source // page, source % page].clone()
            rows[to // page, to % page] = moved


def _exact_tree(case, s):
    if work(case)["flops"] > 1e12:
        return None
    page, Hkv, G, D, w = case["page"], case["heads_kv"], case["heads"] // case["heads_kv"], case["head_dim"], case["window"]
    start, length, parent = s["start"].tolist(), s["length"].tolist(), s["parent"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    at = torch.zeros(s["q"].shape[0], dtype=torch.int32)
    for b, m in enumerate(length):
        first, n = start[b], start[b + 1] - start[b]
        if m < n:
            continue
        base = m - n
        hidden = np.ones((n, m), bool)
        for i in range(n):
            line = [i]
            while parent[first + line[-1]] >= 0:
                line.append(parent[first + line[-1]])
            p = base + len(line) - 1
            at[first + i] = p
            hidden[i, (max(0, p - w + 1) if w else 0):base] = False
            hidden[i, [base + x for x in (line[:w] if w else line)]] = False
        hidden = torch.from_numpy(hidden).cuda()
        used = s["table"][b, :-(-m // page)].long()
        for h in range(Hkv):
            k = s["k_pages"][used, h].reshape(-1, D)[:m].double()
            v = s["v_pages"][used, h].reshape(-1, D)[:m].double()
            z = torch.einsum("tgd,jd->tgj", s["q"][first:first + n, h * G:(h + 1) * G].double(), k) / D ** 0.5
            z = z.masked_fill(hidden[:, None], -math.inf)
            lse[first:first + n, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
            out[first:first + n, h * G:(h + 1) * G] = torch.einsum("tgj,jd->tgd", torch.softmax(z, -1), v)
    return out, lse, at.cuda()


def _exact_sample(s):
    """Row by row, with Python's whole numbers where sums are weighed."""
    l = np.array(s["logits"].float().cpu().numpy(), np.float32)
    l[np.isnan(l)] = -np.inf
    R, V = l.shape
    t, k, p, m = (np.broadcast_to(s[x].cpu().numpy() if isinstance(s[x], torch.Tensor) else np.asarray(s[x]), (R,))
                  for x in ("temperature", "top_k", "top_p", "min_p"))
    u, f32, tokens = s["u"].cpu().numpy(), np.float32, []
    for r in range(R):
        x = l[r]
        top = x.max()
        w = np.zeros(V, np.int64)
        w[x == top] = 0 if top == -np.inf else 1 << 38
        if t[r] > 0:
            lower = np.flatnonzero((x < top) & (x > -np.inf))
            a = np.minimum((top - x[lower]) * (f32(_LOG2E) / f32(t[r])), f32(64))
            n = np.rint(a)
            f = a - n
            y = np.full_like(f, f32(_EXP[6]))
            for c in _EXP[5::-1]:
                y = y * f + f32(c)
            w[lower] = np.floor(np.minimum(np.ldexp(y.astype(np.float64), 38 - n.astype(np.int64)), 2.0 ** 38))
        order = np.lexsort((np.arange(V), -x.astype(np.float64)))
        if 0 < k[r] < V:
            order = order[:int(k[r])]
        if not t[r] > 0:
            order = order[:1]
        upto = np.concatenate(([0], np.cumsum(w[order])))
        if p[r] < 1:
            share = math.floor(float(f32(max(p[r], 0))) * 2 ** 24) * int(upto[-1])
            order = order[upto[:-1] < max(1, -(-share // 2 ** 24))]
        least = math.floor(min(max(float(f32(m[r])), 0.0), 1.0) * 2 ** 38)
        order = np.sort(order[w[order] >= least])
        upto = np.cumsum(w[order])
        goal = math.floor(float(u[r]) * 2 ** 24) * int(upto[-1]) >> 24
        tokens.append(int(order[np.searchsorted(upto, goal, side="right")]) if upto[-1] > 0 else -1)
    return torch.tensor(tokens, dtype=torch.int32, device="cuda")


def _exact_pages(case, s):
    page, table, ref = case["page"], s["table"].tolist(), s["ref"].tolist()
    before, after = s["before"].tolist(), s["after"].tolist()
    for r, n in zip(s["rows"].tolist(), s["keep"].tolist()):
        for g in range(-(-n // page), len(table[r])):
            if table[r][g] >= 0:
                ref[table[r][g]] -= 1
                table[r][g] = -1
    for a, r, n in zip(s["src"].tolist(), s["rows"].tolist(), s["fork_length"].tolist()):
        for g in range(-(-n // page)):
            table[r][g] = table[a][g]
            if table[r][g] >= 0:
                ref[table[r][g]] += 1
    was, unused = list(ref), [i for i, x in enumerate(ref) if x == 0]
    wanted = [(r, g) for r in range(len(table)) if after[r] > before[r]
              for g in range(before[r] // page, -(-after[r] // page)) if table[r][g] < 0 or was[table[r][g]] > 1]
    pairs, missing = [[-1, -1] for _ in table], max(0, len(wanted) - len(unused))
    k, v = s["k_pages"].double(), s["v_pages"].double()
    for (r, g), x in zip(wanted, unused) if not missing else ():
        old = table[r][g]
        if old >= 0:
            ref[old] -= 1
            if g * page < before[r]:
                pairs[r] = [old, x]
                k[x], v[x] = k[old], v[old]
        table[r][g] = x
        ref[x] += 1
    return tuple(torch.tensor(x, dtype=torch.int32, device="cuda") for x in (pairs, [missing], table, ref)) + (k, v)
