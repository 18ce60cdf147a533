"""Trees of drafted tokens on a GB300 against the float64 oracle: layout, attention, accepted paths.

Tolerances of the attention are those derived in test_gpu_attention.py: what a token sees changes
which terms a sum has, not how it is formed.
"""
import random

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from hashed_gram_embedding_engram_gb300 import DraftTree, SequenceBatch, _lib  # noqa: E402
from oracle import decoding_oracle as O  # noqa: E402
from test_gpu_attention import U, Case, f64  # noqa: E402


def random_parents(rng, n, kind):
    if kind == "chain":
        return [-1] + list(range(n - 1)) if n else []
    if kind == "star":
        return [-1] + [0] * (n - 1) if n else []
    if kind == "roots":
        return [-1] * n
    return [rng.randint(-1, i - 1) if kind == "forest" or i == 0 else rng.randint(max(0, i - 9), i - 1) for i in range(n)]


class TreeCase(Case):
    def __init__(self, *, kind="tree", max_nodes=None, parents=None, **shape):
        super().__init__(causal=True, **shape)
        rng = random.Random(shape.get("seed", 0))
        if parents is None:
            parents = [p for n in self.new for p in random_parents(rng, n, kind)]
        self.parents = np.array(parents, np.int64)
        self.parent = torch.tensor(parents, dtype=torch.int32, device="cuda")
        self.words = (max(max_nodes or 0, max(self.new)) + 31) // 32 or 1
        self.tree = self.build()

    def build(self, **kw):
        return DraftTree(self.plan, self.batch, self.parent, max_nodes=32 * self.words, window=self.window, **kw)

    def attend(self, q=None, tree=None, **kw):
        T, H, D = self.q.shape
        out = torch.full((T, H, D), 7.0, dtype=self.q.dtype, device="cuda")
        lse = torch.full((T, H), 7.0, dtype=torch.float32, device="cuda")
        return self.cache.attend_tree(tree or self.tree, self.q if q is None else q, out=out, lse=lse, **kw)

    def check_layout(self, tree=None):
        tree = tree or self.tree
        sees, positions = O.layout(self.parents, self.start, self.length, self.window, 32 * self.words)
        assert tree.positions.cpu().tolist() == positions.tolist()
        bits = tree.mask.cpu().numpy().view(np.uint32)
        for b, n in enumerate(self.new):
            got = (bits[self.start[b]:self.start[b + 1], :, None] >> np.arange(32, dtype=np.uint32) & 1).astype(bool)
            got = got.reshape(n, 32 * self.words)
            assert (got[:, :n] == sees[b][:, :got.shape[1]]).all() and not got[:, n:].any()
        return sees, positions

    def check_tree(self, out, lse, sees=None, positions=None):
        p = self.plan
        if sees is None:
            sees, positions = O.layout(self.parents, self.start, self.length, self.window, 32 * self.words)
        scale = p.scale or p.head_dim ** -0.5
        ref, ref_lse, mag = O.tree_attention(f64(self.q), self.k.double().numpy(), self.v.double().numpy(), self.start,
                                             self.length, self.table, scale, sees, positions, self.window)
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
    # few rows: a single token, small trees, text of none, one and around pages and steps
    dict(new=(1,), length=(1,)),
    dict(new=(1, 2, 3, 4), length=(1, 2, 20, 68)),
    dict(new=(5, 3, 7), length=(68, 66, 135), kind="star"),
    dict(new=(7, 8), length=(64, 1000), D=128, heads=8, heads_kv=2, page=64, kind="forest"),
    dict(new=(16, 9), length=(129, 700), D=128, heads=2, heads_kv=1, page=32),
    dict(new=(31, 32, 30), length=(31, 64, 95), heads=2, heads_kv=2, D=64),
    # more tokens than the launch was told: the same kernel takes further tiles
    dict(new=(33, 40, 1), length=(100, 40, 300), heads=4, heads_kv=1, D=64, hint=2),
    # idle slots, empty sequences, rows that see nothing
    dict(new=(4, 3, 0, 2), length=(0, 2, 9, 30)),
    dict(new=(0, 0, 6, 0), length=(0, 5, 6, 7), kind="roots"),
    # chunks: the word borders of the mask, steps of 128 keys, row tiles
    dict(new=(26,), length=(543,), heads=8, heads_kv=2, D=128, page=16),
    dict(new=(64, 63, 65, 1), length=(64, 200, 128, 129), heads=8, heads_kv=2, D=128, page=64),
    dict(new=(128, 127), length=(500, 127), heads=4, heads_kv=2, D=64, page=32, kind="chain"),
    dict(new=(256, 255, 33), length=(300, 1000, 34), heads=2, heads_kv=2, D=128, page=128),
    dict(new=(200, 7), length=(456, 4000), heads=3, heads_kv=1, D=64, page=32, kind="forest"),
    # windows between positions: of one key, shorter and longer than the tree is deep, over the text
    dict(new=(9, 30), length=(40, 300), window=1),
    dict(new=(40, 20), length=(200, 20), window=3, kind="chain", D=128, heads=8, heads_kv=2),
    dict(new=(64, 50), length=(900, 130), window=70, D=128, heads=4, heads_kv=1, page=32),
    dict(new=(33,), length=(64,), window=4096),
    # other head sizes
    dict(new=(12, 70), length=(77, 100), D=96, heads=6, heads_kv=3),
    dict(new=(1, 40), length=(500, 90), D=256, heads=4, heads_kv=1, page=64, window=50),
    dict(new=(2,), length=(19,), D=8, heads=2, heads_kv=1, page=8),
    dict(new=(3, 5), length=(300, 6), heads=128, heads_kv=1, D=64),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=[str(i) for i in range(len(SHAPES))])
def test_layout_and_attention_match_float64(shape, dtype):
    shape = dict(shape)
    hint = shape.pop("hint", None)
    c = TreeCase(dtype=dtype, seed=11, **shape)
    if hint:
        c.batch = SequenceBatch(c.batch.start, c.batch.length, c.batch.table, max_new=hint)
        c.tree = c.build()
    c.check_layout()
    c.check_tree(*c.attend())


@pytest.mark.parametrize("new,window", [(9, 0), (40, 0), (40, 90)])
def test_a_tile_for_every_block_and_more(new, window):
    """160 and more tiles, which the tiles kernel joins itself (fewer have a kernel of their own for that)."""
    r = np.random.RandomState(new)
    n = r.randint(1, new + 1, 41).tolist()
    c = TreeCase(seed=new, heads=16, heads_kv=4, D=64, page=16, new=n, length=[x + int(m) for x, m in zip(n, r.randint(0, 400, 41))],
                 window=window)
    assert 41 * 4 >= 160 and max(n) * 4 > 32
    a = c.attend()
    c.check_tree(*a)
    b = c.attend()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("shape", [dict(new=(5, 3), length=(80, 40)), dict(new=(60, 40), length=(300, 77), D=128, heads=8)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_chain_is_the_causal_mask(shape, dtype):
    """The same keys and formula.  Not the same bits: a causal tile ends at its last row's key, a tree's
    at the sequence's, so the steps are cut among the blocks at other places and the sums rounded in
    another order.  Each is within its bounds of the one float64 answer."""
    c = TreeCase(dtype=dtype, seed=2, kind="chain", **shape)
    sees, positions = c.check_layout()
    assert all((x == np.tril(np.ones_like(x))).all() for x in sees)
    c.check(*c.run())
    c.check_tree(*c.attend(), sees, positions)


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("f32", 64), ("bf16", 96)])
@pytest.mark.parametrize("new", [(6, 4), (50, 40)])
def test_any_mask_and_stale_slots(dtype, D, new):
    """A mask that is no tree's: random bits, rows that do not see themselves (no key), bits past the
    last token (ignored); infinities and NaN past the length."""
    for stale in (float("nan"), float("inf")):
        c = TreeCase(dtype=dtype, seed=3, new=new, length=(new[0] + 37, new[1] + 200), D=D, stale=stale)
        g = torch.Generator().manual_seed(9)
        bits = torch.randint(-2 ** 31, 2 ** 31, c.tree.mask.shape, generator=g).to(torch.int32)
        c.tree.mask.copy_(bits)
        words = bits.numpy().view(np.uint32)
        sees = []
        for b, n in enumerate(new):
            rows = words[c.start[b]:c.start[b + 1], :, None] >> np.arange(32, dtype=np.uint32) & 1
            sees.append(rows.reshape(n, -1)[:, :n].astype(bool))
        c.check_tree(*c.attend(), sees, f64(c.tree.positions))


def test_positions_before_the_texts_end_count_as_it():
    c = TreeCase(seed=4, new=(20, 3), length=(320, 100), window=40, D=128, heads=8)
    sees, positions = c.check_layout()
    c.tree.positions.fill_(-5)
    c.check_tree(*c.attend(), sees, np.full(23, -5))


@pytest.mark.parametrize("shape", [dict(new=(4, 4), length=(20, 30)), dict(new=(40, 50), length=(90, 300))])
def test_bad_parents_are_reported_and_see_nothing(shape):
    for bad in (-2, 3, 4, 2 ** 31 - 1, -2 ** 31):
        parents = [-1, 0, 1, bad] + [3] + [4] * (shape["new"][0] - 5) if shape["new"][0] > 4 else [-1, 0, 1, bad]
        parents += [-1] + [0] * (shape["new"][1] - 1)
        c = TreeCase(seed=5, parents=parents, **shape)
        assert c.plan.get_error()[0] == _lib.ERR_INDEX_RANGE
        sees, positions = c.check_layout()
        assert not sees[0][3].any() and sees[0][2].any()
        c.check_tree(*c.attend(), sees, positions)


def test_too_many_tokens_for_the_mask_are_reported_and_see_nothing():
    c = TreeCase(seed=6, new=(33, 4), length=(60, 40))
    tree = DraftTree(c.plan, c.batch, c.parent, max_nodes=32)
    assert c.plan.get_error()[0] == _lib.ERR_INDEX_RANGE
    assert not tree.mask[:33].any() and not tree.positions[:33].any() and tree.mask[33:].any()
    out, lse = c.attend(tree=tree)
    assert (out[:33] == 0).all() and torch.isneginf(lse[:33]).all() and torch.isfinite(lse[33:]).all()
    assert c.plan.get_error()[0] == _lib.OK


@pytest.mark.parametrize("new", [(5, 3), (70, 30)])
def test_rows_of_no_sequence_are_left_as_they_were(new):
    """A batch of fixed size whose last rows belong to nobody."""
    c = TreeCase(seed=7, new=new, length=(90, 200))
    T, pad = sum(new), 9
    parent = torch.cat((c.parent, torch.full((pad,), 77, dtype=torch.int32, device="cuda")))
    q = torch.cat((c.q, torch.full((pad, *c.q.shape[1:]), float("nan"), dtype=c.q.dtype, device="cuda")))
    mask = torch.full((T + pad, c.words), 5, dtype=torch.int32, device="cuda")
    at = torch.full((T + pad,), 6, dtype=torch.int32, device="cuda")
    tree = DraftTree(c.plan, c.batch, parent, max_nodes=32 * c.words, mask=mask, positions=at)
    assert tree.mask is mask and (mask[T:] == 5).all() and (at[T:] == 6).all()
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    c.cache.attend_tree(tree, q, out=out, lse=lse)
    assert (out[T:] == 7).all() and (lse[T:] == 7).all()
    c.check_tree(out[:T], lse[:T])


@pytest.mark.parametrize("shape", [dict(new=(3, 2), length=(40, 200)), dict(new=(64, 40), length=(140, 600), D=128, heads=8)])
def test_bad_page_ids_and_lengths(shape):
    c = TreeCase(seed=8, **shape)
    out0, _ = c.attend()
    table, rows = c.batch.table, slice(c.new[0], None)
    for bad in (-1, c.kd.shape[0], 2 ** 31 - 1):
        keep = int(table[0, 1])
        table[0, 1] = bad
        out, _ = c.attend()
        assert c.plan.get_error()[0] == _lib.ERR_INDEX_RANGE
        assert torch.equal(out[rows], out0[rows]) and torch.isfinite(out).all()
        table[0, 1] = keep
    for bad in (10 ** 9, -5):
        c.batch.length[1] = bad
        tree = c.build()
        out, lse = c.attend(tree=tree)
        assert c.plan.get_error()[0] == _lib.ERR_INDEX_RANGE
        assert not tree.mask[rows].any() and (out[rows] == 0).all() and torch.isneginf(lse[rows]).all()


def test_strided_queries_and_the_same_bits_every_time():
    c = TreeCase(seed=9, new=(20, 60), length=(50, 200), heads=8, heads_kv=2, D=128, page=32)
    a = c.attend()
    T, H, D = c.q.shape
    packed = torch.full((T, H + 4, D), float("nan"), dtype=c.q.dtype, device="cuda")
    packed[:, 2:H + 2] = c.q
    for q in (packed[:, 2:H + 2], c.q.transpose(0, 1).contiguous().transpose(0, 1), c.q):
        b = c.attend(q=q, workspace=c.plan.new_workspace())
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_graph_replay_reads_the_trees_of_the_day():
    c = TreeCase(seed=10, new=(20, 12, 30), length=(300, 41, 77), heads=8, heads_kv=2, D=128, page=32)
    out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:2], device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.build()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            tree = c.build()
            c.cache.attend_tree(tree, c.q, out=out, lse=lse)
    torch.cuda.current_stream().wait_stream(s)
    rng = random.Random(1)
    for length in ([300, 41, 77], [250, 12, 11], [20, 0, 64]):
        c.length = length
        c.batch.length.copy_(torch.tensor(length, dtype=torch.int32))
        c.parents = np.array([p for n in c.new for p in random_parents(rng, n, "forest")])
        c.parent.copy_(torch.from_numpy(c.parents))
        graph.replay()
        torch.cuda.synchronize()
        c.check_layout(tree)
        c.check_tree(out, lse)


def test_calls_on_two_streams_and_replays_beside_them():
    """Tiles cut into parts on each of two streams, and a captured call replayed on a third: a workspace each."""
    cases = [TreeCase(seed=20 + i, new=(40, 64), length=(3000, 2500), heads=8, heads_kv=2, D=128, page=32) for i in range(3)]
    for c in cases[1:]:                                 # one plan, three caches
        c.plan = cases[0].plan
        c.cache = type(c.cache)(c.plan, c.kd, c.vd)
        c.tree = c.build()
    want = [c.attend() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(streams[2]):
        with torch.cuda.graph(graph, stream=streams[2]):
            replayed = cases[2].cache.attend_tree(cases[2].tree, cases[2].q)
    got = []
    for _ in range(20):
        for c, s in zip(cases[:2], streams):
            with torch.cuda.stream(s):
                got.append((c, c.cache.attend_tree(c.tree, c.q)))
        with torch.cuda.stream(streams[2]):
            graph.replay()
    torch.cuda.synchronize()
    for c, (out, lse) in got + [(cases[2], replayed)]:
        o, l = want[cases.index(c)]
        assert torch.equal(out, o) and torch.equal(lse, l)


# ---------------------------------------------------------------- accepted paths
def accept_case(seed, B, most, vocab, width):
    rng = random.Random(seed)
    new = [rng.randint(0, most) for _ in range(B)]
    start = np.concatenate(([0], np.cumsum(new))).astype(np.int64)
    length = [0 if rng.random() < 0.1 else n + rng.randint(0, 50) for n in new]
    T = int(start[-1])
    parents = [p for n in new for p in random_parents(rng, n, rng.choice(("tree", "chain", "star", "forest")))]
    tokens, sampled = ([rng.randrange(vocab) for _ in range(T)] for _ in range(2))
    return start, length, parents, tokens, sampled


@pytest.mark.parametrize("B,most,vocab,width", [(1, 1, 2, 1), (5, 9, 1, 3), (40, 70, 2, 16), (3, 256, 1, 256),
                                                (2, 700, 1, 200), (300, 20, 3, 8)])
def test_accepted_paths(B, most, vocab, width):
    start, length, parents, tokens, sampled = accept_case(B + most, B, most, vocab, width)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    c = Case(new=(1,), length=(1,))
    table = torch.zeros(B, 60, dtype=torch.int32, device="cuda")
    tree = DraftTree(c.plan, SequenceBatch(i32(start), i32(length), table), i32(parents), max_nodes=256)
    c.plan.get_error()                              # of trees too large for a mask, which the walk does not need
    got = tree.accept(i32(tokens), i32(sampled), width=width)
    want = O.accept(parents, tokens, sampled, start, length, width)
    for x, y in zip(got, want):
        assert x.cpu().tolist() == y.tolist()
    assert c.plan.get_error()[0] == _lib.OK


def test_no_tokens_and_no_sequences():
    c = Case(new=(1,), length=(1,))
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    batch = SequenceBatch(zero, torch.tensor([0, 5], dtype=torch.int32, device="cuda"), zero[:2].view(2, 1))
    tree = DraftTree(c.plan, batch, z)
    path, count, emitted, length = tree.accept(z, z, width=2)
    assert (path == -1).all() and (emitted == -1).all() and count.tolist() == [0, 0] and length.tolist() == [0, 5]
    assert c.cache.attend_tree(tree, c.q[:0])[0].shape[0] == 0
    none = DraftTree(c.plan, SequenceBatch(zero[:1], z, z.view(0, 1)), z)
    assert none.accept(z, z)[0].shape == (0, 16)
    c.cache.attend_tree(none, c.q[:0])
    assert c.plan.get_error()[0] == _lib.OK
