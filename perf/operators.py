"""Cases and plain forms of the attention sub-block's serving operators.

qk_norm_rope   per-head RMSNorm of queries and keys with the position rotation
kv_append      keys (normalised, rotated) and values into a paged cache, the queries in the same call
attend         attention of a chunk of new tokens, or of single tokens, over the paged cache
verify         drafted tokens against the target's probabilities, from given random numbers
"""
import math
import random

import torch

own = False

# the layer widths this repository works with, as heads: d = 1024 (8 x 128 or 16 x 64), d = 4096 (32 x 128)
_HEADS = ((8, 2, 128), (16, 4, 64), (32, 8, 128))
_VOCAB = 129280
_EPS = 1e-6


def listed():
    return [
        # one decode step of 256 sequences, d = 1024
        dict(name="norm_rope_decode", op="norm_rope", dtype="bf16", T=256, heads=8, heads_kv=2, head_dim=128,
             rotary=128, style="halves", norm=True, rope_len=8192),
        # an fp32 prefill of 4 x 4096 tokens and one, half of each head rotated, adjacent pairs
        dict(name="norm_rope_prefill_f32", op="norm_rope", dtype="f32", T=16385, heads=16, heads_kv=4, head_dim=64,
             rotary=32, style="adjacent", norm=True, rope_len=20000),
        # a decode step of 256 sequences into their caches
        dict(name="append_decode", op="append", dtype="bf16", B=256, heads=8, heads_kv=2, head_dim=128, page=16,
             rotary=128, style="halves", norm=True, new_min=1, new_max=1, len_min=1, len_max=1000),
        # chunks of unequal length of 8 sequences, d = 4096
        dict(name="append_chunks", op="append", dtype="bf16", B=8, heads=32, heads_kv=8, head_dim=128, page=64,
             rotary=128, style="halves", norm=True, new_min=1, new_max=4096, len_min=1, len_max=8192),
        # one interactive sequence, early in its answer: latency
        dict(name="attend_decode_one", op="attend", dtype="bf16", B=1, heads=8, heads_kv=2, head_dim=128, page=16,
             new_min=1, new_max=1, len_min=517, len_max=517, causal=True, window=0, idle=0),
        # the decode batch of 256 sequences at unequal lengths, some slots idle
        dict(name="attend_decode_batch", op="attend", dtype="bf16", B=256, heads=32, heads_kv=8, head_dim=128, page=16,
             new_min=1, new_max=1, len_min=1, len_max=4096, causal=True, window=0, idle=3),
        # few sequences with long contexts: the keys have to be split over the SMs
        dict(name="attend_decode_long", op="attend", dtype="bf16", B=3, heads=32, heads_kv=8, head_dim=128, page=64,
             new_min=1, new_max=1, len_min=30011, len_max=131072, causal=True, window=0, idle=0),
        # drafted tokens: several rows a sequence over its cache
        dict(name="attend_drafts", op="attend", dtype="bf16", B=32, heads=32, heads_kv=8, head_dim=128, page=64,
             new_min=1, new_max=6, len_min=100, len_max=8192, causal=True, window=0, idle=0),
        # a prefill chunk of 4096 tokens behind 4096 earlier ones
        dict(name="attend_prefill", op="attend", dtype="bf16", B=1, heads=32, heads_kv=8, head_dim=128, page=64,
             new_min=4096, new_max=4096, len_min=8192, len_max=8192, causal=True, window=0, idle=0),
        # fp32 layers: ragged chunks with a sliding window
        dict(name="attend_window_f32", op="attend", dtype="f32", B=5, heads=16, heads_kv=4, head_dim=64, page=32,
             new_min=1, new_max=700, len_min=700, len_max=2500, causal=True, window=512, idle=0),
        # one sequence's three drafts against the framework's vocabulary
        dict(name="verify_one", op="verify", dtype="f32", B=1, S=3, V=_VOCAB, draft_probs=True),
        # the decode batch, five drafts each
        dict(name="verify_batch", op="verify", dtype="f32", B=256, S=5, V=_VOCAB, draft_probs=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw(rng):
    op = rng.choice(("norm_rope", "append", "attend", "attend", "attend", "verify"))
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    heads, heads_kv, head_dim = rng.choice(_HEADS)
    heads_kv = rng.choice([h for h in (1, heads_kv, heads_kv * 2, heads) if heads % h == 0 and heads // h <= 16])
    rope = dict(rotary=rng.choice((head_dim, head_dim // 2)), style=rng.choice(("halves", "adjacent")),
                norm=rng.random() < 0.75)
    shape = dict(heads=heads, heads_kv=heads_kv, head_dim=head_dim)
    if op == "norm_rope":
        return dict(op=op, dtype=dtype, T=_log_int(rng, 1, 16385), rope_len=rng.choice((4096, 8192, 20000)),
                    **shape, **rope)
    if op == "verify":
        return dict(op=op, dtype=dtype, B=_log_int(rng, 1, 256), S=rng.randint(1, 8),
                    V=rng.choice((_VOCAB, _log_int(rng, 1000, 200000))), draft_probs=rng.random() < 0.7)
    page = rng.choice((16, 32, 64, 128))
    if op == "append":
        new_max = rng.choice((1, _log_int(rng, 2, 4096)))
        return dict(op=op, dtype=dtype, B=_log_int(rng, 1, 256 if new_max == 1 else 8), page=page,
                    new_min=1, new_max=new_max, len_min=1, len_max=_log_int(rng, new_max, 8192), **shape, **rope)
    kind = rng.choice(("decode", "decode", "drafts", "chunk"))
    window = rng.choice((0, 0, 0, _log_int(rng, 16, 4096)))
    causal = rng.random() < 0.9
    if kind == "chunk":
        new_max = _log_int(rng, 8, 4096 if dtype == "bf16" else 700)
        B, len_max = _log_int(rng, 1, 8), _log_int(rng, new_max, 16384 if dtype == "bf16" else 2500)
        new_min = rng.choice((1, new_max))
    else:
        new_max = 1 if kind == "decode" else rng.randint(2, 8)
        B, len_max, new_min = _log_int(rng, 1, 256), _log_int(rng, 16, 131072), 1
    return dict(op=op, dtype=dtype, B=B, page=page, new_min=new_min, new_max=new_max,
                len_min=rng.randint(new_max, len_max), len_max=len_max, causal=causal, window=window,
                idle=rng.choice((0, 0, 1)) if B > 1 else 0, **shape)


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    """A case of the listed ranges that costs no more than the largest listed one, and whose plain form's scores,
    padded over the batch, stay under 8 GB."""
    while True:
        case = _draw(rng)
        padded = 1
        if case["op"] == "attend":
            padded = case["B"] * case["len_max"] * max(case["heads"] * case["new_max"],
                                                       case["heads_kv"] * case["head_dim"])
        limit = 2e9 if case["dtype"] == "f32" and case["op"] == "attend" else 4e9
        if padded <= 2 ** 31 and _cost(case) <= limit:
            return case


# ---------------------------------------------------------------- what a case's sequences are
def _spread(lo, hi, n, salt):
    """n whole numbers over [lo, hi], both ends among them where n > 1, in an order of their own."""
    v = [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]
    random.Random(salt).shuffle(v)
    return v


def _sequences(case):
    """(new tokens, tokens in the cache after the chunk) of each sequence; idle slots have a row and no tokens."""
    new = _spread(case["new_min"], case["new_max"], case["B"], 3)
    length = [max(a, b) for a, b in zip(new, _spread(case["len_min"], case["len_max"], case["B"], 5))]
    for b in range(case.get("idle", 0)):
        length[(b * 7 + 1) % case["B"]] = 0
    return new, length


def _size(case):
    return 4 if case["dtype"] == "f32" else 2


def _torch_type(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def work(case):
    op, e = case["op"], _size(case)
    if op == "verify":
        # row a of the target; after a rejection (about one draft in four is turned down) row a of the draft too
        rejected = 1 - 0.75 ** case["S"]
        rows = case["B"] * (1 + (rejected if case["draft_probs"] else 0))
        return dict(bytes=rows * case["V"] * e, flops=2 * rows * case["V"])
    H, Hkv, D = case["heads"], case["heads_kv"], case["head_dim"]
    if op == "norm_rope":
        n = case["T"] * (H + Hkv) * D
        return dict(bytes=2 * n * e + case["T"] * (4 * case["rotary"] + 4), flops=9 * n)
    new, length = _sequences(case)
    if op == "append":
        T = sum(new)
        return dict(bytes=2 * T * (H + 2 * Hkv) * D * e + 4 * T * case["rotary"], flops=9 * T * (H + Hkv) * D)
    keys = pairs = 0
    w = case["window"]
    for n, m in zip(new, length):
        lo = max(0, m - n - w + 1) if w else 0
        keys += max(0, m - lo)
        for i in range(n):
            p = m - n + i
            hi = min(m, p + 1) if case["causal"] else m
            pairs += max(0, hi - (max(0, p - w + 1) if w else 0)) if p >= 0 else 0
    T = sum(new)
    return dict(bytes=keys * Hkv * D * 2 * e + T * H * (2 * D * e + 4), flops=4 * pairs * H * D)


# ---------------------------------------------------------------- inputs
def _rope_table(length, rotary):
    """[length, rotary]: cosines of the rotary/2 angles, then their sines."""
    inv = 10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda") / rotary)
    angle = torch.arange(length, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat((angle.cos(), angle.sin()), 1).float()


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)
    dt, op = _torch_type(case), case["op"]

    def normal(*shape):
        out = torch.empty(shape, dtype=dt, device="cuda")
        return out.normal_(generator=g)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    if op == "verify":
        B, S, V = case["B"], case["S"], case["V"]
        logits = torch.randn((B, S + 1, V), generator=g, device="cuda") * 4
        draft = logits[:, :S] + 0.5 * torch.randn((B, S, V), generator=g, device="cuda")
        gumbel = -torch.log(-torch.log(uniform(B, S, V).clamp_(1e-7, 1 - 1e-6)))
        drafts = (draft + gumbel).argmax(-1).to(torch.int32)
        del gumbel
        target = torch.softmax(logits, -1).to(dt)
        del logits
        probs = torch.softmax(draft, -1).to(dt) if case["draft_probs"] else None
        n = torch.randint(0, S + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        n[: (B + 1) // 2] = S
        return dict(target=target, probs=probs, drafts=drafts, n_drafts=n, u=uniform(B, S + 1))
    H, Hkv, D = case["heads"], case["heads_kv"], case["head_dim"]
    s = {}
    if op in ("norm_rope", "append"):
        # queries, keys and values as the views of one projection's output
        T = case["T"] if op == "norm_rope" else sum(_sequences(case)[0])
        qkv = normal(T, H + 2 * Hkv, D)
        s.update(q=qkv[:, :H], k=qkv[:, H:H + Hkv], v=qkv[:, H + Hkv:], g_q=None, g_k=None)
        if case["norm"]:
            s.update(g_q=1 + 0.1 * torch.randn(D, generator=g, device="cuda"),
                     g_k=1 + 0.1 * torch.randn(D, generator=g, device="cuda"))
        if op == "norm_rope":
            s["positions"] = torch.randint(0, case["rope_len"], (T,), generator=g, device="cuda", dtype=torch.int32)
            s["rope"] = _rope_table(case["rope_len"], case["rotary"])
            return s
    new, length = _sequences(case)
    page = case["page"]
    per = max(1, (max(length) + page - 1) // page)
    used = [(m + page - 1) // page for m in length]
    pages = sum(used) + 1
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((case["B"], per), dtype=torch.int32, device="cuda")
    at = 0
    for b, m in enumerate(used):
        table[b, :m] = order[at:at + m]
        at += m
    start = [0]
    for m in new:
        start.append(start[-1] + m)
    s.update(start=torch.tensor(start, dtype=torch.int32, device="cuda"),
             length=torch.tensor(length, dtype=torch.int32, device="cuda"), table=table,
             k_pages=normal(pages, Hkv, page, D), v_pages=normal(pages, Hkv, page, D))
    if op == "append":
        s["rope"] = _rope_table(max(length), case["rotary"])
    else:
        s["q"] = normal(start[-1], H, D)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        import hashed_gram_embedding_engram_gb300 as E
        s["E"] = E
        if case["op"] == "verify":
            B, S = case["B"], case["S"]
            s["tokens"] = torch.empty((B, S + 1), dtype=torch.int32, device="cuda")
            s["accepted"] = torch.empty((B,), dtype=torch.int32, device="cuda")
            return s
        s["plan"] = E.AttentionPlan(heads=case["heads"], heads_kv=case["heads_kv"], head_dim=case["head_dim"],
                                    page=case.get("page", 64), dtype=case["dtype"], rotary_dim=case.get("rotary", 0),
                                    rope_style=case.get("style", "halves"), eps=_EPS)
        s["q_out"] = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
        if case["op"] == "norm_rope":
            s["k_out"] = torch.empty(s["k"].shape, dtype=s["k"].dtype, device="cuda")
        else:
            s["cache"] = E.PagedCache(s["plan"], s["k_pages"], s["v_pages"])
            s["batch"] = E.SequenceBatch(s["start"], s["length"], s["table"], max_new=case["new_max"])
            if case["op"] == "attend":
                s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    return s


def run(s):
    op = s["case"]["op"]
    if op == "verify":
        return _own_verify(s) if own else _plain_verify(s)
    if op == "norm_rope":
        if own:
            return s["plan"].qk_norm_rope(s["q"], s["k"], s["positions"], s["rope"], g_q=s["g_q"], g_k=s["g_k"],
                                          q_out=s["q_out"], k_out=s["k_out"])
        return _plain_norm_rope(s["q"], s["g_q"], s), _plain_norm_rope(s["k"], s["g_k"], s)
    if op == "append":
        if own:
            s["cache"].append(s["batch"], s["k"], s["v"], rope=s["rope"], g_k=s["g_k"], q=s["q"], g_q=s["g_q"],
                              q_out=s["q_out"])
            return s["q_out"], s["k_pages"], s["v_pages"]
        return _plain_append(s)
    if own:
        return s["cache"].attend(s["batch"], s["q"], causal=s["case"]["causal"], window=s["case"]["window"],
                                 out=s["q_out"], lse=s["lse"])
    return _plain_attend(s)


# ---------------------------------------------------------------- plain forms
def _own_verify(s):
    return s["E"].verify_drafts(s["target"], s["drafts"], s["u"], draft_probs=s["probs"], n_drafts=s["n_drafts"],
                                tokens=s["tokens"], accepted=s["accepted"])


def _plain_norm_rope(x, g, s):
    case = s["case"]
    y = x.float()
    if g is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + _EPS) * g
    r = case["rotary"]
    row = s["rope"][s["positions"].long()][:, None]
    cos, sin = row[..., :r // 2], row[..., r // 2:]
    if case["style"] == "halves":
        a, c = y[..., :r // 2], y[..., r // 2:r]
        turned = torch.cat((a * cos - c * sin, a * sin + c * cos), -1)
    else:
        a, c = y[..., :r:2], y[..., 1:r:2]
        turned = torch.stack((a * cos - c * sin, a * sin + c * cos), -1).flatten(-2)
    return torch.cat((turned, y[..., r:]), -1).to(x.dtype)


def _plain_rows(s, T):
    """The sequence and the position of each of the T packed rows."""
    row = torch.arange(T, device="cuda")
    b = torch.searchsorted(s["start"].long(), row, right=True) - 1
    return b, s["length"].long()[b] - s["start"].long()[b + 1] + row


def _plain_append(s):
    page = s["case"]["page"]
    b, p = _plain_rows(s, s["q"].shape[0])
    turned = dict(s, positions=p)
    at = s["table"].long()[b, p // page]
    s["k_pages"][at, :, p % page] = _plain_norm_rope(s["k"], s["g_k"], turned)
    s["v_pages"][at, :, p % page] = s["v"]
    return _plain_norm_rope(s["q"], s["g_q"], turned), s["k_pages"], s["v_pages"]


def _plain_attend(s):
    case, q = s["case"], s["q"]
    H, Hkv, D, page = case["heads"], case["heads_kv"], case["head_dim"], case["page"]
    B, N, T, L = case["B"], case["new_max"], q.shape[0], s["table"].shape[1] * case["page"]
    start, length = s["start"].long(), s["length"].long()
    new = start[1:] - start[:-1]
    i = torch.arange(N, device="cuda")
    rows = (start[:-1, None] + i).clamp(max=T - 1)
    x = q[rows].float().view(B, N, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    table = s["table"].long()
    k = s["k_pages"][table].transpose(1, 2).reshape(B, Hkv, L, D).float()
    score = torch.matmul(x, k.transpose(2, 3)).mul_(1 / math.sqrt(D)).view(B, Hkv, H // Hkv, N, L)
    del k
    j, p = torch.arange(L, device="cuda"), (length - new)[:, None] + i
    seen = (j < length[:, None, None]) & (p >= 0)[:, :, None]
    if case["causal"]:
        seen = seen & (j <= p[:, :, None])
    if case["window"]:
        seen = seen & (j > p[:, :, None] - case["window"])
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = score.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    v = s["v_pages"][table].transpose(1, 2).reshape(B, Hkv, L, D).float()
    out = torch.matmul(e.view(B, Hkv, -1, L), v).view(B, Hkv, H // Hkv, N, D)
    out = out / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + total.log()).squeeze(-1)
    b, at = _plain_rows(s, T)
    at = at - (length - new)[b]
    out = out.permute(0, 3, 1, 2, 4).reshape(B, N, H, D)[b, at]
    return out.to(q.dtype), lse.permute(0, 3, 1, 2).reshape(B, N, H)[b, at]


def _fixed(x):
    return (torch.nan_to_num(x.float(), nan=0.0).clamp(0, 1) * 2.0 ** 38).to(torch.int64)


def _plain_verify(s):
    p, x, S = s["target"], s["drafts"].long(), s["case"]["S"]
    n, u = s["n_drafts"].long(), (s["u"].clamp(0, 1 - 2.0 ** -24) * 2.0 ** 24).to(torch.int64)
    px = _fixed(p[:, :S].gather(2, x[..., None]).squeeze(-1))
    qx = torch.full_like(px, 2 ** 38) if s["probs"] is None else _fixed(s["probs"].gather(2, x[..., None]).squeeze(-1))
    i = torch.arange(S, device="cuda")
    ok = (u[:, :S] * qx < px * 2 ** 24) & (i < n[:, None])
    a = ok.long().cumprod(1).sum(1)
    each = torch.arange(p.shape[0], device="cuda")
    w = _fixed(p[each, a])
    last = a.clamp(max=S - 1)
    if s["probs"] is None:
        drafted = torch.zeros_like(w).scatter_(1, x[each, last][:, None], 2 ** 38)
    else:
        drafted = _fixed(s["probs"][each, last])
    left = (w - drafted).clamp(min=0)
    turned = (a < n) & (left.sum(1) > 0)
    w = torch.where(turned[:, None], left, w)
    upto = w.cumsum(1)
    total, v = upto[:, -1], u[:, S]
    goal = v * (total >> 24) + ((v * (total & (2 ** 24 - 1))) >> 24)
    following = (upto <= goal[:, None]).sum(1)
    following = torch.where(total > 0, following, torch.full_like(following, -1))
    k = torch.arange(S + 1, device="cuda")
    kept = torch.cat((x, x[:, :1]), 1)
    tokens = torch.where(k < a[:, None], kept, torch.full_like(kept, -1))
    tokens = torch.where(k == a[:, None], following[:, None], tokens)
    return tokens.to(torch.int32), a.to(torch.int32)


# ---------------------------------------------------------------- the definitions in 64 bits
def _turn64(x, g, table, at, case):
    y = x.double()
    if g is not None:
        y = y / ((y ** 2).sum(-1, keepdim=True) / y.shape[-1] + _EPS).sqrt() * g.double()
    out, r = y.clone(), case["rotary"]
    for m in range(r // 2):
        c, z = table[at, m].double()[:, None], table[at, r // 2 + m].double()[:, None]
        lo, hi = (m, m + r // 2) if case["style"] == "halves" else (2 * m, 2 * m + 1)
        out[..., lo] = y[..., lo] * c - y[..., hi] * z
        out[..., hi] = y[..., hi] * c + y[..., lo] * z
    return out


def exact(case, seed):
    s, op = _inputs(case, seed), case["op"]
    if op == "norm_rope":
        at = s["positions"].long()
        return _turn64(s["q"], s["g_q"], s["rope"], at, case), _turn64(s["k"], s["g_k"], s["rope"], at, case)
    if op == "verify":
        return _exact_verify(case, s)
    new, length = _sequences(case)
    page, Hkv, G, D = case["page"], case["heads_kv"], case["heads"] // case["heads_kv"], case["head_dim"]
    if op == "append":
        at = torch.cat([torch.arange(m - n, m, device="cuda") for n, m in zip(new, length)])
        q, k = _turn64(s["q"], s["g_q"], s["rope"], at, case), _turn64(s["k"], s["g_k"], s["rope"], at, case)
        kp, vp, first = s["k_pages"].double(), s["v_pages"].double(), 0
        for b, (n, m) in enumerate(zip(new, length)):
            for t in range(-(-n // page) + 1):  # the pieces of the chunk that lie in one page
                lo, hi = max(m - n, ((m - n) // page + t) * page), min(m, ((m - n) // page + t + 1) * page)
                if lo < hi:
                    rows, where = slice(first + lo - (m - n), first + hi - (m - n)), int(s["table"][b, lo // page])
                    kp[where, :, lo % page:lo % page + hi - lo] = k[rows].transpose(0, 1)
                    vp[where, :, lo % page:lo % page + hi - lo] = s["v"][rows].double().transpose(0, 1)
            first += n
        return q, kp, vp
    if work(case)["flops"] > 1e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    first = 0
    for b, (n, m) in enumerate(zip(new, length)):
        used = s["table"][b, :-(-m // page)].long()
        for h in range(Hkv if m else 0):
            k = s["k_pages"][used, h].reshape(-1, D)[:m].double()
            v = s["v_pages"][used, h].reshape(-1, D)[:m].double()
            for r in range(0, n, 512):
                rows = slice(first + r, first + min(n, r + 512))
                at = torch.arange(m - n + r, m - n + min(n, r + 512), device="cuda")[:, None]
                j = torch.arange(m, device="cuda")[None]
                hidden = torch.zeros((at.shape[0], m), dtype=torch.bool, device="cuda")
                if case["causal"]:
                    hidden |= j > at
                if case["window"]:
                    hidden |= j <= at - case["window"]
                z = torch.einsum("tgd,jd->tgj", s["q"][rows, h * G:(h + 1) * G].double(), k) / D ** 0.5
                z = z.masked_fill(hidden[:, None], -math.inf)
                lse[rows, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
                out[rows, h * G:(h + 1) * G] = torch.einsum("tgj,jd->tgd", torch.softmax(z, -1).nan_to_num(0.0), v)
        first += n
    return out, lse


def _exact_verify(case, s):
    """With Python's whole numbers for the tests and NumPy-free 64-bit sums for the rows."""
    B, S = case["B"], case["S"]
    tokens, accepted = torch.full((B, S + 1), -1, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    drafts, n, u = s["drafts"].cpu().tolist(), s["n_drafts"].cpu().tolist(), s["u"].double().cpu().tolist()
    for b in range(B):
        a = 0
        while a < n[b]:
            x = drafts[b][a]
            p = math.floor(float(s["target"][b, a, x]) * 2 ** 38)
            q = 2 ** 38 if s["probs"] is None else math.floor(float(s["probs"][b, a, x]) * 2 ** 38)
            if not math.floor(u[b][a] * 2 ** 24) * q < p * 2 ** 24:
                break
            tokens[b, a], a = x, a + 1
        w = torch.floor(s["target"][b, a].double() * 2 ** 38).long()
        if a < n[b]:
            q = torch.zeros_like(w)
            if s["probs"] is None:
                q[drafts[b][a]] = 2 ** 38
            else:
                q = torch.floor(s["probs"][b, a].double() * 2 ** 38).long()
            rest = torch.relu(w - q)
            w = rest if int(rest.sum()) else w
        goal = math.floor(u[b][S] * 2 ** 24) * int(w.sum()) // 2 ** 24
        tokens[b, a] = int(torch.searchsorted(w.cumsum(0), goal, right=True))
        accepted[b] = a
    return tokens.cuda(), accepted.cuda()
