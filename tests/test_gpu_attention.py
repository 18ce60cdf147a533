"""Attention over the paged cache, the append, norm and rotation, and the draft check on a
GB300, against the float64 oracle.

Tolerances (derived, u = 2^-24 the unit round-off of binary32, A = sum softmax |v|):
 * bf16 out: one rounding of the output (2^-8 |out|: bf16 has 8 significant bits) and one of
   each weight (2^-8 A), and the float part below.
 * float part: a score is a D-term float sum, off by at most (D + 4) u S with S = the largest
   scale sum |q||k| of the case, so a weight is off by twice that, plus L u for the sum over L
   keys and 2^-20 for the exponential: (2 (D + 4) u S + L u + 2^-20) A.
 * lse: (D + 4) u S + L u + 2^-20 (1 + |lse|).
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from hashed_gram_embedding_engram_gb300 import (AttentionPlan, EngramError, PagedCache, SequenceBatch, _lib,  # noqa: E402
                                                verify_drafts)
from oracle import attention_oracle as O  # noqa: E402

U = 2.0 ** -24


def f64(t):
    return t.double().cpu().numpy()


class Case:
    """Seeded inputs: pages in a shuffled order, every slot no sequence uses filled with `stale`."""

    def __init__(self, *, dtype="bf16", heads=4, heads_kv=2, D=64, page=16, new=(1,), length=(17,), causal=True,
                 window=0, seed=0, stale=float("nan"), scale=None, spread=1.0, extra_pages=3):
        g = torch.Generator().manual_seed(seed)
        self.plan = AttentionPlan(heads=heads, heads_kv=heads_kv, head_dim=D, page=page, dtype=dtype, rotary_dim=0,
                                  scale=scale)
        dt = self.plan.torch_dtype
        self.new, self.length, self.page, self.causal, self.window = list(new), list(length), page, causal, window
        self.start = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
        B, used = len(new), [-(-m // page) for m in length]
        pages, per = sum(used) + extra_pages, max(1, max(used))
        order = torch.randperm(pages, generator=g).numpy().astype(np.int32)
        self.table = np.full((B, per), -1, np.int32)      # entries past a length are never used
        live = torch.zeros(pages, page, dtype=torch.bool)
        at = 0
        for b, m in enumerate(used):
            self.table[b, :m] = order[at:at + m]
            at += m
            for j in range(length[b]):
                live[self.table[b, j // page], j % page] = True
        shape = (pages, heads_kv, page, D)
        self.k = (torch.randn(shape, generator=g) * spread).to(dt)
        self.v = torch.randn(shape, generator=g).to(dt)
        self.live = live[:, None, :, None].expand(shape)
        self.kd = torch.where(self.live, self.k, torch.tensor(stale, dtype=dt)).cuda()
        self.vd = torch.where(self.live, self.v, torch.tensor(stale, dtype=dt)).cuda()
        self.q = (torch.randn(int(self.start[-1]), heads, D, generator=g) * spread).to(dt).cuda()
        self.cache = PagedCache(self.plan, self.kd, self.vd)
        self.batch = SequenceBatch(torch.from_numpy(self.start).cuda(), torch.tensor(length, dtype=torch.int32).cuda(),
                                   torch.from_numpy(self.table).cuda(), max_new=max(new))

    def run(self, q=None, **kw):
        T, H, D = self.q.shape
        out = torch.full((T, H, D), 7.0, dtype=self.q.dtype, device="cuda")
        lse = torch.full((T, H), 7.0, dtype=torch.float32, device="cuda")
        return self.cache.attend(self.batch, self.q if q is None else q, causal=self.causal, window=self.window,
                                 out=out, lse=lse, **kw)

    def check(self, out, lse):
        p = self.plan
        scale = p.scale or p.head_dim ** -0.5
        ref, ref_lse, mag = O.attention(f64(self.q), self.k.double().numpy(), self.v.double().numpy(), self.start,
                                        self.length, self.table, scale, self.causal, self.window)
        out, lse = f64(out), f64(lse)
        S = scale * p.head_dim * float(self.q.abs().max()) * float(self.k.abs().max()) * 0.5
        L = max(self.length) + 1
        bound = (2 * (p.head_dim + 4) * U * S + L * U + 2.0 ** -20) * mag + 1e-30
        if p.dtype == "bf16":
            bound = bound + 2.0 ** -8 * np.abs(ref) + 2.0 ** -8 * mag
        worst = (np.abs(out - ref) / bound).max() if out.size else 0
        assert np.isfinite(out).all() and worst <= 1.0, f"out {worst:.3g} of its bound"
        empty = np.isneginf(ref_lse)
        assert np.array_equal(np.isneginf(lse), empty)
        assert (out[empty] == 0).all()
        tol = (p.head_dim + 4) * U * S + L * U + 2.0 ** -20 * (1 + np.abs(ref_lse[~empty]))
        assert (np.abs(lse[~empty] - ref_lse[~empty]) <= tol).all()
        st, flags = p.get_error()
        assert st == _lib.OK, (st, flags)


SHAPES = [
    # one token: lengths of 1, at and around a page, a tile and many tiles
    dict(new=(1,), length=(1,)),
    dict(new=(1,) * 6, length=(1, 15, 16, 17, 33, 130)),
    dict(new=(1,) * 3, length=(511, 1, 257), heads=8, heads_kv=1, D=128, page=32),
    dict(new=(1, 1), length=(4099, 3000), heads=8, heads_kv=8, D=128, page=64),
    dict(new=(1,), length=(6001,), heads=16, heads_kv=2, D=64, page=16),
    # idle slots, rows without keys, sequences without new tokens
    dict(new=(1, 1, 1, 1), length=(0, 20, 0, 3)),
    dict(new=(0, 3, 0, 0, 2, 0), length=(9, 3, 0, 40, 1, 5)),
    dict(new=(5, 4), length=(2, 0)),
    # a few tokens (drafts), odd groups
    dict(new=(3, 6, 1), length=(100, 6, 259), heads=12, heads_kv=4, D=128, page=64),
    dict(new=(7, 2), length=(300, 77), heads=10, heads_kv=2, D=64, page=8),
    dict(new=(2, 5), length=(150, 1000), heads=32, heads_kv=1, D=128, page=128),
    # chunks: from the start, behind earlier tokens, ragged, across row tiles
    dict(new=(70,), length=(70,)),
    dict(new=(129, 1, 40), length=(129, 333, 1000), heads=4, heads_kv=2, D=128, page=64),
    dict(new=(300, 17), length=(700, 17), heads=8, heads_kv=2, D=128, page=16),
    dict(new=(513,), length=(1300,), heads=2, heads_kv=2, D=128, page=256),
    dict(new=(260, 255), length=(260, 900), heads=3, heads_kv=1, D=64, page=32),
    # without the causal mask
    dict(new=(33, 1), length=(100, 50), causal=False),
    dict(new=(300,), length=(400,), causal=False, D=128, heads=4, heads_kv=1, page=64),
    # windows: of one key, inside a tile, across tiles, longer than the sequence
    dict(new=(1, 1), length=(300, 5), window=1),
    dict(new=(40, 1), length=(200, 999), window=7),
    dict(new=(200, 90), length=(600, 90), window=150, D=128, heads=8, heads_kv=2, page=32),
    dict(new=(20,), length=(64,), window=4096),
    dict(new=(30,), length=(90,), window=13, causal=False),
    # other head sizes
    dict(new=(1, 20), length=(77, 50), D=96, heads=6, heads_kv=3),
    dict(new=(1, 70), length=(500, 90), D=256, heads=4, heads_kv=1, page=64),
    dict(new=(2,), length=(19,), D=8, heads=2, heads_kv=1, page=8),
    # all heads one group of 128, and large scores
    dict(new=(1, 2), length=(300, 5), heads=128, heads_kv=1, D=64),
    dict(new=(9, 1), length=(200, 600), spread=6.0, D=128, heads=8, heads_kv=2),
    dict(new=(5,), length=(40,), scale=0.01),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=[str(i) for i in range(len(SHAPES))])
def test_attention_matches_float64(shape, dtype):
    c = Case(dtype=dtype, seed=11, **shape)
    c.check(*c.run())


@pytest.mark.parametrize("stale", [float("inf"), -3e38, 1e30])
def test_slots_past_the_length_are_not_read_into_the_result(stale):
    for shape in (dict(new=(1, 1), length=(17, 130)), dict(new=(200, 9), length=(213, 77), D=128, page=64)):
        c = Case(seed=3, stale=stale, **shape)
        c.check(*c.run())


@pytest.mark.parametrize("shape", [SHAPES[4], SHAPES[13]])
def test_same_bits_every_time_and_with_any_workspace(shape):
    c = Case(seed=5, **shape)
    a = c.run()
    ws = c.plan.new_workspace()
    for _ in range(3):
        b = c.run(workspace=ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_queries(dtype):
    """Queries as views: of a packed projection's output, and of a head-major array."""
    c = Case(seed=6, dtype=dtype, new=(5, 130), length=(50, 200), heads=8, heads_kv=2, D=128, page=32)
    a = c.run()
    T, H, D = c.q.shape
    packed = torch.full((T, H + 4, D), float("nan"), dtype=c.q.dtype, device="cuda")
    packed[:, :H] = c.q
    major = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    for q in (packed[:, :H], major):
        b = c.run(q=q)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_nan_and_infinity_in_visible_keys_stay_in_their_sequence():
    c = Case(seed=7, new=(1, 1, 1), length=(50, 60, 300), D=128, heads=8, heads_kv=2)
    a = c.run()
    c.kd[int(c.table[1, 0]), 0, 3, 5] = float("nan")
    b = c.run()
    assert torch.isnan(b[0][1, :4]).all() and torch.isnan(b[1][1, :4]).all()
    keep = torch.ones(3, 8, dtype=torch.bool, device="cuda")
    keep[1, :4] = False
    assert torch.equal(a[0][keep], b[0][keep]) and torch.equal(a[1][keep], b[1][keep])


def test_a_score_of_minus_infinity_is_a_key_without_weight():
    """A whole row of -inf scores has no weight at all: out 0, lse -inf."""
    c = Case(seed=8, new=(1, 1), length=(40, 40), heads=2, heads_kv=1, D=64)
    c.q.fill_(1.0)
    c.kd[c.table[0, :3].tolist()] = torch.where(c.live[c.table[0, :3].tolist()].cuda(), -torch.inf, c.kd[c.table[0, :3].tolist()])
    out, lse = c.run()
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()
    assert torch.isfinite(out[1]).all() and torch.isfinite(lse[1]).all()


@pytest.mark.parametrize("shape", [dict(new=(1, 1), length=(40, 200)), dict(new=(140, 1), length=(140, 60), D=128)])
def test_bad_page_ids_and_lengths_are_reported_and_not_read(shape):
    c = Case(seed=9, **shape)
    out0, _ = c.run()
    table = c.batch.table
    for bad in (-1, c.kd.shape[0], 2 ** 31 - 1, -2 ** 31):
        keep = int(table[0, 1])
        table[0, 1] = bad
        out, _ = c.run()
        st, _ = c.plan.get_error()
        assert st == _lib.ERR_INDEX_RANGE
        rows = slice(c.new[0], None)
        assert torch.equal(out[rows], out0[rows])       # the other sequence is as it was
        assert torch.isfinite(out).all()
        table[0, 1] = keep
    c.batch.length[1] = 10 ** 9
    c.run()
    assert c.plan.get_error()[0] == _lib.ERR_INDEX_RANGE
    c.batch.length[1] = -5
    out, lse = c.run()
    assert c.plan.get_error()[0] == _lib.ERR_INDEX_RANGE
    assert (out[c.new[0]:] == 0).all() and torch.isneginf(lse[c.new[0]:]).all()
    c.batch.length[1] = c.length[1]
    c.check(*c.run())


def test_starts_outside_the_rows_are_reported_and_not_followed():
    c = Case(seed=10, new=(2, 3), length=(20, 30))
    c.batch.start.copy_(torch.tensor([0, 2, 900], dtype=torch.int32))
    c.run()
    assert c.plan.get_error()[0] == _lib.ERR_INDEX_RANGE
    c.batch.start.copy_(torch.tensor([-4, 2, 1], dtype=torch.int32))
    c.run()
    assert c.plan.get_error()[0] == _lib.ERR_INDEX_RANGE


def test_graph_replay_reads_the_lengths_of_the_day():
    c = Case(seed=12, new=(1, 1, 1), length=(300, 41, 77), heads=8, heads_kv=2, D=128, page=32)
    ws = c.plan.new_workspace()
    out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:2], device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.cache.attend(c.batch, c.q, out=out, lse=lse, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            c.cache.attend(c.batch, c.q, out=out, lse=lse, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    for length in ([300, 41, 77], [12, 41, 0], [299, 1, 64]):
        c.length = length
        c.batch.length.copy_(torch.tensor(length, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        c.check(out, lse)


def test_calls_on_two_streams_use_two_workspaces():
    cases = [Case(seed=20 + i, new=(1,) * 4, length=(900, 2000, 77, 4000), heads=8, heads_kv=2, D=128, page=32) for i in range(2)]
    cases[1].plan = cases[0].plan                       # one plan, two caches, two streams
    cases[1].cache = PagedCache(cases[0].plan, cases[1].kd, cases[1].vd)
    want = [c.run() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(20):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append((c, c.cache.attend(c.batch, c.q)))
    torch.cuda.synchronize()
    for c, (out, lse) in got:
        o, l = want[cases.index(c)]
        assert torch.equal(out, o) and torch.equal(lse, l)


def test_offsets_past_32_bits():
    """Pages whose elements, and bytes, lie past 2^32."""
    plan = AttentionPlan(heads=8, heads_kv=8, head_dim=128, page=64, rotary_dim=0)
    pages = 2 ** 32 // (8 * 64 * 128) + 40
    cache = PagedCache.empty(plan, pages)
    cache.k[-8:].normal_()
    cache.v[-8:].normal_()
    g = torch.Generator(device="cuda").manual_seed(1)
    for new in (1, 150):
        length = 64 * 5 + 9
        table = torch.arange(pages - 6, pages, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
        start = torch.tensor([0, new], dtype=torch.int32, device="cuda")
        n = torch.tensor([length], dtype=torch.int32, device="cuda")
        k = torch.randn(new, 8, 128, generator=g, device="cuda").bfloat16()
        v = torch.randn(new, 8, 128, generator=g, device="cuda").bfloat16()
        q = torch.randn(new, 8, 128, generator=g, device="cuda").bfloat16()
        batch = SequenceBatch(start, n, table, max_new=new)
        cache.append(batch, k, v)
        out, lse = cache.attend(batch, q)
        small = AttentionPlan(heads=8, heads_kv=8, head_dim=128, page=64, rotary_dim=0)
        near = PagedCache(small, cache.k[-6:].clone(), cache.v[-6:].clone())
        batch2 = SequenceBatch(start, n, table - (pages - 6), max_new=new)
        want, want_lse = near.attend(batch2, q)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        rows = torch.arange(length - new, length)
        for j in rows[:: max(1, new // 7)].tolist():
            assert torch.equal(cache.k[int(table[0, j // 64]), :, j % 64], k[j - (length - new)])
    assert plan.get_error()[0] == _lib.OK


def test_no_tokens_and_no_sequences():
    c = Case(seed=13, new=(0, 0), length=(5, 3))
    out, lse = c.run()
    assert out.shape[0] == 0
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    batch = SequenceBatch(torch.zeros(1, dtype=torch.int32, device="cuda"), z, z.view(0, 1), max_new=0)
    out, lse = c.cache.attend(batch, c.q[:0])
    assert out.shape[0] == 0
    c.cache.append(batch, c.q[:0, :2], c.q[:0, :2])
    assert c.plan.get_error()[0] == _lib.OK


# ---------------------------------------------------------------- norm, rotation, append
def rope_inputs(dtype, heads, heads_kv, D, T, seed):
    g = torch.Generator().manual_seed(seed)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    qkv = torch.randn(T, heads + 2 * heads_kv, D, generator=g).to(dt).cuda()
    gq, gk = (1 + 0.1 * torch.randn(D, generator=g)).cuda(), (1 + 0.1 * torch.randn(D, generator=g)).cuda()
    return qkv[:, :heads], qkv[:, heads:heads + heads_kv], qkv[:, heads + heads_kv:], gq, gk


def assert_rope(got, ref, dtype, what):
    """Float arithmetic: the norm's sum of D terms, a quotient, three products and a sum, each
    within 2^-24: 2^-19 of the pair's size (at most sqrt(2) of the larger element is hidden in
    the factor); bf16 adds one rounding, 2^-8 of the value."""
    got = f64(got)
    size = np.sqrt((ref ** 2).max(-1, keepdims=True))
    bound = 2.0 ** -19 * size + (2.0 ** -8 * 1.001 * np.abs(ref) if dtype == "bf16" else 0) + 1e-30
    worst = (np.abs(got - ref) / bound).max()
    assert worst <= 1.0, f"{what}: {worst:.3g} of its bound"


ROPE = [dict(heads=4, heads_kv=2, D=64, r=64), dict(heads=8, heads_kv=2, D=128, r=128),
        dict(heads=5, heads_kv=1, D=128, r=32), dict(heads=3, heads_kv=3, D=96, r=48), dict(heads=2, heads_kv=1, D=256, r=256),
        dict(heads=2, heads_kv=2, D=8, r=0), dict(heads=32, heads_kv=8, D=128, r=64), dict(heads=7, heads_kv=1, D=40, r=16)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("style", ["halves", "adjacent"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("shape", ROPE, ids=[str(i) for i in range(len(ROPE))])
def test_qk_norm_rope_matches_float64(shape, norm, style, dtype):
    H, Hkv, D, r = shape["heads"], shape["heads_kv"], shape["D"], shape["r"]
    for T in (1, 37, 300):
        q, k, _, gq, gk = rope_inputs(dtype, H, Hkv, D, T, 3 + T)
        plan = AttentionPlan(heads=H, heads_kv=Hkv, head_dim=D, dtype=dtype, rotary_dim=r, rope_style=style)
        rope = plan.rope_table(500) if r else None
        pos = torch.randint(0, 500, (T,), dtype=torch.int32, generator=torch.Generator().manual_seed(T)).cuda()
        g = (gq, gk) if norm else (None, None)
        qo, ko = plan.qk_norm_rope(q, k, pos if r else None, rope, g_q=g[0], g_k=g[1])
        for got, x, w in ((qo, q, g[0]), (ko, k, g[1])):
            ref = O.norm_rope(f64(x), None if w is None else f64(w), plan.eps, pos.cpu().numpy(),
                              None if rope is None else rope.cpu().numpy(), style == "adjacent")
            assert_rope(got, ref, dtype, f"T={T}")
        only, none = plan.qk_norm_rope(q, None, pos if r else None, rope, g_q=g[0])
        assert none is None and torch.equal(only, qo)
        dense = q.contiguous()
        plan.qk_norm_rope(dense, None, pos if r else None, rope, g_q=g[0], q_out=dense)   # in place
        assert torch.equal(dense, qo)
        assert plan.get_error()[0] == _lib.OK


def test_positions_outside_the_table_are_reported_and_not_rotated():
    q, k, _, gq, gk = rope_inputs("bf16", 4, 2, 64, 6, 1)
    plan = AttentionPlan(heads=4, heads_kv=2, head_dim=64)
    rope = plan.rope_table(50)
    pos = torch.tensor([0, 49, 50, -1, 2 ** 31 - 1, 7], dtype=torch.int32, device="cuda")
    qo, ko = plan.qk_norm_rope(q, k, pos, rope, g_q=gq, g_k=gk)
    assert plan.get_error()[0] == _lib.ERR_INDEX_RANGE
    ref = O.norm_rope(f64(q), f64(gq), plan.eps, pos.cpu().numpy(), rope.cpu().numpy())
    assert_rope(qo, ref, "bf16", "q")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("style", ["halves", "adjacent"])
@pytest.mark.parametrize("shape", [
    dict(heads=4, heads_kv=2, D=64, r=64, page=16, new=(1,) * 5, length=(1, 16, 17, 0, 300)),
    dict(heads=8, heads_kv=2, D=128, r=128, page=64, new=(70, 0, 1, 130), length=(70, 3, 64, 500)),
    dict(heads=6, heads_kv=3, D=96, r=32, page=8, new=(9, 4), length=(5, 100)),
    dict(heads=2, heads_kv=1, D=256, r=256, page=128, new=(1, 2), length=(129, 2)),
    dict(heads=1, heads_kv=1, D=8, r=0, page=8, new=(3,) * 600, length=tuple(range(600))),
], ids=["decode", "chunks", "padding", "wide", "many"])
def test_append_matches_float64_and_touches_nothing_else(shape, style, dtype):
    H, Hkv, D, r, page = (shape[n] for n in ("heads", "heads_kv", "D", "r", "page"))
    new, length = shape["new"], shape["length"]
    start = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    T = int(start[-1])
    q, k, v, gq, gk = rope_inputs(dtype, H, Hkv, D, T, 9)
    plan = AttentionPlan(heads=H, heads_kv=Hkv, head_dim=D, page=page, dtype=dtype, rotary_dim=r, rope_style=style)
    rope = plan.rope_table(max(length) + 1) if r else None
    used = [-(-m // page) for m in length]
    pages = sum(used) + 2
    order = np.random.RandomState(4).permutation(pages).astype(np.int32)
    table = np.full((len(new), max(used)), -1, np.int32)
    at = 0
    for b, m in enumerate(used):
        table[b, :m] = order[at:at + m]
        at += m
    cache = PagedCache.empty(plan, pages)
    cache.k.fill_(3.0)
    cache.v.fill_(5.0)
    batch = SequenceBatch(torch.from_numpy(start).cuda(), torch.tensor(length, dtype=torch.int32).cuda(),
                          torch.from_numpy(table).cuda(), max_new=max(new))
    qo = cache.append(batch, k, v, rope, g_k=gk, q=q, g_q=gq)
    assert plan.get_error()[0] == _lib.OK
    pos = O.positions(start, length)
    tab = None if rope is None else rope.cpu().numpy()
    ref_k = O.norm_rope(f64(k), f64(gk), plan.eps, pos, tab, style == "adjacent")
    assert_rope(qo, O.norm_rope(f64(q), f64(gq), plan.eps, pos, tab, style == "adjacent"), dtype, "q")
    kp, vp = cache.k.clone(), cache.v.clone()
    t_at, p_at, s_at = [], [], []
    for b in range(len(new)):
        for i in range(new[b]):
            p = length[b] - new[b] + i
            if p >= 0:
                t_at.append(start[b] + i), p_at.append(int(table[b, p // page])), s_at.append(p % page)
    assert_rope(kp[p_at, :, s_at], ref_k[t_at], dtype, "k")
    assert torch.equal(vp[p_at, :, s_at], v[t_at])
    kp[p_at, :, s_at], vp[p_at, :, s_at] = 3.0, 5.0
    assert (kp == 3).all() and (vp == 5).all()
    again = cache.append(batch, k, v, rope, g_k=gk)       # without queries: the same cache
    assert again is None
    assert_rope(cache.k[p_at, :, s_at], ref_k[t_at], dtype, "k")


def test_append_reports_bad_pages_and_writes_nothing_there():
    plan = AttentionPlan(heads=2, heads_kv=1, head_dim=64, page=16, rotary_dim=0)
    cache = PagedCache.empty(plan, 4)
    cache.k.fill_(1)
    cache.v.fill_(1)
    _, k, v, _, _ = rope_inputs("bf16", 2, 1, 64, 3, 2)
    start = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    length = torch.tensor([1, 33, 40], dtype=torch.int32, device="cuda")
    table = torch.tensor([[4, 0], [0, 1], [-7, 1]], dtype=torch.int32, device="cuda")   # 33 and 40: past two pages
    cache.append(SequenceBatch(start, length, table, max_new=1), k, v)
    assert plan.get_error()[0] == _lib.ERR_INDEX_RANGE
    assert (cache.k == 1).all() and (cache.v == 1).all()


def test_append_then_attend_equals_attention_over_the_same_keys():
    """A prefill in chunks and single tokens gives the rows of one prefill."""
    plan = AttentionPlan(heads=8, heads_kv=2, head_dim=128, page=32)
    T, g = 200, torch.Generator().manual_seed(2)
    qkv = torch.randn(T, 12, 128, generator=g).bfloat16().cuda()
    rope = plan.rope_table(T)
    table = torch.randperm(9, generator=g)[:7].to(torch.int32)[None].cuda().contiguous()

    def steps(cuts):
        cache, outs = PagedCache.empty(plan, 9), []
        for lo, hi in zip(cuts[:-1], cuts[1:]):
            x = qkv[lo:hi]
            batch = SequenceBatch(torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda"),
                                  torch.tensor([hi], dtype=torch.int32, device="cuda"), table, max_new=hi - lo)
            q = cache.append(batch, x[:, 8:10], x[:, 10:], rope, q=x[:, :8])
            outs.append(cache.attend(batch, q)[0])
        return torch.cat(outs).float()

    whole = steps([0, T])
    for cuts in ([0, 64, 65, 66, 130, T], [0, 1, 2, 100, T]):
        parts = steps(cuts)
        # both are within 2^-8 (|out| + A) of the same reals, A <= max |v| < 5
        assert (whole - parts).abs().max() <= 2 * 2.0 ** -8 * 2 * 5
        assert (whole - parts).norm() <= 5e-3 * whole.norm()


# ---------------------------------------------------------------- draft check
def draft_inputs(B, S, V, seed, dtype=torch.float32, certain=False):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(B, S + 1, V, generator=g) * 3
    noisy = logits[:, :S] + 0.7 * torch.randn(B, S, V, generator=g)
    target, draft = torch.softmax(logits, -1).to(dtype), torch.softmax(noisy, -1).to(dtype)
    drafts = torch.multinomial(draft.float().view(B * S, V), 1, generator=g).view(B, S).to(torch.int32)
    return target, None if certain else draft, drafts, torch.rand(B, S + 1, generator=g)


def check_verify(target, draft, drafts, n, u):
    t, a = verify_drafts(target.cuda(), drafts.cuda(), u.cuda(), draft_probs=None if draft is None else draft.cuda(),
                         n_drafts=None if n is None else n.cuda())
    want_t, want_a = O.verify(target.float().numpy(), None if draft is None else draft.float().numpy(), drafts.numpy(),
                              None if n is None else n.numpy(), u.numpy())
    assert np.array_equal(a.cpu().numpy(), want_a) and np.array_equal(t.cpu().numpy(), want_t)
    return t, a


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("B,S,V", [(1, 1, 1), (3, 2, 5), (40, 5, 257), (17, 3, 4096), (5, 8, 10007), (2, 64, 33),
                                   (3, 40, 1000), (4, 4, 129280)])
def test_verify_equals_whole_numbers(B, S, V, certain, dtype):
    for seed in range(3):
        target, draft, drafts, u = draft_inputs(B, S, V, seed, dtype, certain)
        check_verify(target, draft, drafts, None, u)
        n = torch.randint(-1, S + 3, (B,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
        check_verify(target, draft, drafts, n, u)


def test_verify_edges():
    V, S = 1000, 2
    target, draft, drafts, u = draft_inputs(6, S, V, 5)
    for value in (0.0, 1.0, 1 - 2.0 ** -24, float("nan"), -1.0, 2.0, 2.0 ** -30):
        check_verify(target, draft, drafts, None, torch.full_like(u, value))
    out = drafts.clone()
    out[0, 0], out[1, 1], out[2, 0] = -1, V, 2 ** 31 - 1           # no such token: turned down
    check_verify(target, draft, out, None, u)
    check_verify(target, None, out, None, u)
    same = target[:, :S].clone()                                    # p = q: always kept, the rest is 0
    check_verify(target, same, drafts, None, u)
    certain = torch.zeros_like(target)
    certain[:, :, 7] = 1.0
    check_verify(certain, draft, torch.full_like(drafts, 7), None, u)
    t, a = check_verify(certain, None, torch.full_like(drafts, 3), None, u)
    assert (t[:, 0] == 7).all() and (a == 0).all()
    zero = torch.zeros_like(target)
    t, a = check_verify(zero, draft, drafts, None, u)
    assert (t == -1).all()
    bad = target.clone()
    bad[:, :, ::3], bad[:, :, 1], bad[:, :, 4] = float("nan"), float("inf"), -1.0
    check_verify(bad, draft, drafts, None, u)
    tiny = torch.full_like(target, 2.0 ** -39)                      # below the fixed point's last place
    tiny[:, :, 500] = 2.0 ** -38
    t, _ = check_verify(tiny, None, drafts, torch.zeros(6, dtype=torch.int32), u)
    assert (t[:, 0] == 500).all()
    p_less = target[:, :S] * 1.5                                    # p <= q everywhere: the rest is 0, p itself is used
    check_verify(target, p_less, drafts, None, torch.full_like(u, 0.99))


# ---------------------------------------------------------------- refusals
def test_refusals_of_the_front_end():
    c = Case(seed=1, new=(2,), length=(9,))
    q = c.q
    with pytest.raises(TypeError):
        c.cache.attend(c.batch, q.float())
    with pytest.raises(ValueError):
        c.cache.attend(c.batch, q.cpu())
    with pytest.raises(ValueError):
        c.cache.attend(c.batch, q[:, :3])
    with pytest.raises(ValueError):
        c.cache.attend(c.batch, q.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(EngramError, match="INVALID_ARG"):
        c.cache.attend(c.batch, q, window=-1)
    with pytest.raises(EngramError, match="WORKSPACE"):
        c.cache.attend(c.batch, q, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(EngramError, match="INVALID_ARG"):
        wide = torch.zeros(2, 4, 65, dtype=q.dtype, device="cuda")   # head stride of 130 bytes
        c.cache.attend(c.batch, wide[:, :, :64])
    with pytest.raises(EngramError, match="INVALID_ARG"):
        flat = torch.zeros(2 * 4 * 64 + 1, dtype=q.dtype, device="cuda")[1:]
        c.cache.attend(c.batch, flat.view(2, 4, 64))
    with pytest.raises(ValueError):
        SequenceBatch(c.batch.start, c.batch.length, c.batch.table[0])
    with pytest.raises(TypeError):
        SequenceBatch(c.batch.start.long(), c.batch.length, c.batch.table)
    with pytest.raises(ValueError):
        PagedCache(c.plan, c.kd[:, :, :8], c.vd[:, :, :8])
    for bad in (dict(heads=3, heads_kv=2), dict(head_dim=12), dict(head_dim=264), dict(page=24), dict(page=4),
                dict(rotary_dim=24), dict(rotary_dim=80), dict(eps=0.0)):
        with pytest.raises(EngramError, match="INVALID_ARG"):
            AttentionPlan(**{**dict(heads=4, heads_kv=2, head_dim=64), **bad})
    plan = AttentionPlan(heads=4, heads_kv=2, head_dim=64, page=16)
    with pytest.raises(EngramError, match="INVALID_ARG"):
        plan.qk_norm_rope(q)                                          # rotation asked for, no table
    with pytest.raises(ValueError):
        plan.qk_norm_rope(q, None, torch.zeros(2, dtype=torch.int32, device="cuda"), plan.rope_table(9)[:, :32])
    p = torch.zeros(2, 3, 10, device="cuda")
    d, u = torch.zeros(2, 2, dtype=torch.int32, device="cuda"), torch.zeros(2, 3, device="cuda")
    with pytest.raises(ValueError):
        verify_drafts(p.half(), d, u)
    with pytest.raises(ValueError):
        verify_drafts(p, d[:, :1], u)
    with pytest.raises(TypeError):
        verify_drafts(p, d.long(), u)
    with pytest.raises(EngramError, match="INVALID_ARG"):
        verify_drafts(p[:, :1].contiguous(), d[:, :0].contiguous(), u[:, :1].contiguous())


@pytest.mark.parametrize("hint", [1, 5, 40, 0, 10 ** 6])
def test_max_new_is_a_hint_only(hint):
    """Whatever launch the hint picks, every row is computed."""
    c = Case(seed=14, new=(3, 200, 1), length=(40, 333, 1000), heads=8, heads_kv=2, D=128, page=32)
    c.batch = SequenceBatch(c.batch.start, c.batch.length, c.batch.table, max_new=hint)
    c.check(*c.run())


@pytest.mark.parametrize("hint", [1, 2, 200])
def test_pages_outside_a_window_are_not_looked_at(hint):
    """Table entries of pages that no query sees may hold anything (an engine frees them)."""
    c = Case(seed=15, new=(2, 1), length=(600, 131), heads=8, heads_kv=2, D=128, page=16, window=100)
    c.batch = SequenceBatch(c.batch.start, c.batch.length, c.batch.table, max_new=hint)
    table = c.batch.table
    table[0, :(600 - 2 - 100) // 16] = 2 ** 30
    table[1, :(131 - 1 - 99) // 16] = -3
    c.check(*c.run())


def test_capture_on_a_new_stream_leaves_its_later_calls_alone():
    """The first call on a stream is captured; calls on that stream, before and between replays,
    share nothing with the graph."""
    c = Case(seed=16, new=(1, 1), length=(4000, 900), heads=8, heads_kv=2, D=128, page=32)
    want = c.run()
    torch.cuda.synchronize()
    junk = torch.full((1 << 28,), 255, dtype=torch.uint8, device="cuda")     # what a new allocation may hold
    del junk
    out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:2], device="cuda")
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.cache.attend(c.batch, c.q, out=out, lse=lse)
    for _ in range(2):
        with torch.cuda.stream(s):
            got = c.cache.attend(c.batch, c.q)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("D,page", [(64, 32), (128, 64)])
def test_fp32_errors_do_not_grow_with_the_length(D, page):
    """Norm-wise error of a single token over 30000 keys.  Scores of size up to 8 (in powers of two)
    are rounded to 2^-24 of that, 4 2^-24 on average in a weight; a step's sum is a chain of 64
    additions (about sqrt(64) / 2 = 4 roundings of the partial sums' size) and the steps' sums one of
    a few hundred in a block, each again half a rounding: 16 2^-24 = 1e-6 is not reached, where one
    chain over all keys (sqrt(30000) / 2 = 87 roundings) is several times it."""
    c = Case(seed=17, dtype="f32", new=(1,), length=(30000,), heads=4, heads_kv=2, D=D, page=page)
    out, lse = c.run()
    ref, ref_lse, _ = O.attention(f64(c.q), c.k.double().numpy(), c.v.double().numpy(), c.start, c.length, c.table,
                                  D ** -0.5)
    assert np.linalg.norm(f64(out) - ref) <= 16 * U * np.linalg.norm(ref)
    assert np.abs(f64(lse) - ref_lse).max() <= 16 * U * np.abs(ref_lse).max()
