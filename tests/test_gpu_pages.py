"""Pages freed, forked, reserved, copied and compacted on a GB300, against plain Python: whole
numbers and copies, so everything has to be equal."""
import random

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from hashed_gram_embedding_engram_gb300 import AttentionPlan, PagedCache, PagePool, SequenceBatch, _lib  # noqa: E402
from oracle import decoding_oracle as O  # noqa: E402


def i32(x):
    return torch.tensor(np.asarray(x).tolist(), dtype=torch.int32, device="cuda")


def make_plan(page=16, dtype="bf16", heads_kv=2, D=64):
    return AttentionPlan(heads=heads_kv, heads_kv=heads_kv, head_dim=D, page=page, dtype=dtype, rotary_dim=0)


def bits(t):
    return t.view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def random_cache(plan, pages, seed=0):
    """Any bits, NaN and infinities among them: copies do not look at values."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.int32 if plan.dtype == "f32" else torch.int16
    shape = (pages, plan.heads_kv, plan.page, plan.head_dim)
    k, v = (torch.randint(torch.iinfo(dt).min, torch.iinfo(dt).max, shape, generator=g, device="cuda", dtype=dt)
            .view(plan.torch_dtype) for _ in range(2))
    return PagedCache(plan, k, v)


# ---------------------------------------------------------------- copies
@pytest.mark.parametrize("dtype,page,heads_kv,D", [("bf16", 8, 1, 8), ("bf16", 16, 2, 64), ("bf16", 128, 8, 128),
                                                   ("f32", 64, 3, 96), ("f32", 8, 1, 8), ("bf16", 1024, 1, 256)])
def test_pages_are_copied_whole(dtype, page, heads_kv, D):
    plan = make_plan(page, dtype, heads_kv, D)
    cache = random_cache(plan, 12)
    k, v = cache.k.clone(), cache.v.clone()
    pairs = [(0, 5), (-1, 3), (2, -1), (0, 11), (7, 4), (-1, -1), (-2 ** 31, 6)]
    cache.copy_pages(i32(pairs))
    for a, b in pairs:
        if a >= 0 and b >= 0:
            k[b], v[b] = k[a], v[a]
    assert torch.equal(bits(cache.k), bits(k)) and torch.equal(bits(cache.v), bits(v))
    assert plan.get_error()[0] == _lib.OK


def test_pages_past_the_cache_are_reported_and_left_out():
    plan = make_plan()
    cache = random_cache(plan, 4)
    k = cache.k.clone()
    for pair in ((0, 4), (4, 0), (2 ** 31 - 1, 1)):
        cache.copy_pages(i32([pair]))
        assert plan.get_error()[0] == _lib.ERR_INDEX_RANGE
    cache.copy_pages(i32(np.zeros((0, 2))).view(0, 2))
    assert torch.equal(bits(cache.k), bits(k)) and plan.get_error()[0] == _lib.OK


def test_many_pairs():
    plan = make_plan(8, "bf16", 1, 8)
    cache = random_cache(plan, 20000)
    k = cache.k.clone()
    pairs = torch.randperm(20000, generator=torch.Generator().manual_seed(1)).view(-1, 2)
    cache.copy_pages(i32(pairs))
    k[pairs[:, 1].cuda()] = k[pairs[:, 0].cuda()]
    assert torch.equal(bits(cache.k), bits(k))


# ---------------------------------------------------------------- rows moved together
def compact_inputs(seed, length, new, page, keep):
    rng = random.Random(seed)
    used = [-(-m // page) for m in length]
    order = list(range(sum(used) + 2))
    rng.shuffle(order)
    table = np.full((len(length), max(max(used), 1)), -1, np.int64)
    at = 0
    for b, m in enumerate(used):
        table[b, :m] = order[at:at + m]
        at += m
    count = [min(n, round(n * keep)) for n in new]
    path = np.full((len(length), max(max(count), 1) + 2), 123456, np.int64)
    for b, (n, c) in enumerate(zip(new, count)):
        path[b, :c] = sorted(rng.sample(range(n), c))
    return table, path, count, len(order)


COMPACT = [dict(length=(1,), new=(1,), keep=1.0), dict(length=(40, 7, 100), new=(20, 7, 1), keep=0.5),
           dict(length=(300, 0, 65, 12), new=(64, 0, 65, 0), keep=0.1), dict(length=(2000, 999), new=(2000, 999), keep=0.9),
           dict(length=(700, 1500), new=(650, 1500), keep=0.3), dict(length=(513,), new=(513,), keep=1.0)]


@pytest.mark.parametrize("dtype,page,heads_kv,D", [("bf16", 16, 2, 64), ("bf16", 64, 8, 128), ("f32", 32, 3, 96),
                                                   ("bf16", 8, 1, 8), ("f32", 128, 1, 256), ("bf16", 16, 5, 104)])
@pytest.mark.parametrize("shape", COMPACT, ids=[str(i) for i in range(len(COMPACT))])
def test_kept_rows_move_together(shape, dtype, page, heads_kv, D):
    table, path, count, pages = compact_inputs(3, shape["length"], shape["new"], page, shape["keep"])
    plan = make_plan(page, dtype, heads_kv, D)
    cache = random_cache(plan, pages)
    start = np.concatenate(([0], np.cumsum(shape["new"])))
    want = [O.compact(bits(x).cpu().numpy(), table, start, shape["length"], path, count) for x in (cache.k, cache.v)]
    cache.compact(SequenceBatch(i32(start), i32(shape["length"]), i32(table)), i32(path), i32(count))
    assert (bits(cache.k).cpu().numpy() == want[0]).all() and (bits(cache.v).cpu().numpy() == want[1]).all()
    assert plan.get_error()[0] == _lib.OK


def test_paths_that_do_not_ascend_move_nothing_and_are_reported():
    plan = make_plan()
    cache = random_cache(plan, 8)
    before = cache.k.clone()
    start, length = [0, 10, 20], [40, 30]
    table = [[0, 1, 2], [3, 4, -1]]
    batch = SequenceBatch(i32(start), i32(length), i32(table))
    good = [2, 5, 9]
    for path, count in (([3, 3, 4], 3), ([4, 3, 5], 3), ([-1, 3, 4], 3), ([0, 1, 10], 3), (good, 4), (good, -1),
                        (good, 2 ** 31 - 1)):
        cache.k.copy_(before)
        cache.compact(batch, i32([path, good]), i32([count, 3]))
        assert plan.get_error()[0] == _lib.ERR_INDEX_RANGE
        want = O.compact(bits(before).cpu().numpy(), table, start, length, np.array([[0, 1, 2], good]), [0, 3])
        assert (bits(cache.k).cpu().numpy() == want).all()
    # an idle sequence that keeps none is fine; one that would keep some is not
    cache.compact(SequenceBatch(i32(start), i32([0, 30]), i32(table)), i32([good, good]), i32([0, 3]))
    assert plan.get_error()[0] == _lib.OK
    cache.compact(SequenceBatch(i32(start), i32([0, 30]), i32(table)), i32([good, good]), i32([1, 0]))
    assert plan.get_error()[0] == _lib.ERR_INDEX_RANGE


def test_bad_pages_are_left_out_of_a_move():
    plan = make_plan()
    cache = random_cache(plan, 8)
    start, length, path = [0, 40], [40], [[1, 20, 35, 36]]
    for table in ([[0, 1, 8]], [[0, -1, 2]], [[2 ** 31 - 1, 1, 2]]):
        want = O.compact(bits(cache.k).cpu().numpy(), table, start, length, np.array(path), [4])
        cache.compact(SequenceBatch(i32(start), i32(length), i32(table)), i32(path), i32([4]))
        assert plan.get_error()[0] == _lib.ERR_INDEX_RANGE
        assert (bits(cache.k).cpu().numpy() == want).all()


def test_rows_past_32_bits():
    """Slots whose elements lie past 2^32."""
    plan = make_plan(64, "bf16", 8, 128)
    pages = 2 ** 32 // (8 * 64 * 128) + 8
    cache = PagedCache.empty(plan, pages)
    cache.k[-4:].normal_()
    want = cache.k[-2, :, 3:63:10].clone()
    table = i32([[pages - 2, pages - 1]])
    cache.compact(SequenceBatch(i32([0, 128]), i32([128]), table), i32([list(range(3, 63, 10))]), i32([6]))
    assert torch.equal(cache.k[-2, :, :6], want)
    cache.copy_pages(i32([[pages - 2, pages - 4]]))
    assert torch.equal(cache.k[-4], cache.k[-2]) and plan.get_error()[0] == _lib.OK


# ---------------------------------------------------------------- the table
class Both:
    """A pool on the GPU beside one in Python."""

    def __init__(self, rows, table_pages, pages, page=16):
        self.plan = make_plan(page)
        self.pool = PagePool.empty(self.plan, rows, table_pages, pages)
        self.ref = O.Pool(self.pool.table.cpu().numpy(), self.pool.ref.cpu().numpy(), page)

    def same(self, error=False):
        assert self.pool.table.cpu().tolist() == self.ref.table and self.pool.ref.cpu().tolist() == self.ref.ref
        assert (self.plan.get_error()[0] != _lib.OK) == error

    def free(self, rows, keep, error=False):
        self.pool.free(i32(rows), i32(keep))
        self.ref.free(rows, keep)
        self.same(error)

    def fork(self, src, dst, length, error=False):
        self.pool.fork(i32(src), i32(dst), i32(length))
        self.ref.fork(src, dst, length)
        self.same(error)

    def reserve(self, before, after, error=False):
        pairs, missing = self.pool.reserve(i32(before), i32(after))
        want = self.ref.reserve(before, after)
        assert (pairs.cpu().tolist(), missing.tolist()) == (want[0], [want[1]])
        self.same(error)
        return want

    def counted(self):
        """Every page's count is the number of entries that name it."""
        named = [e for r in self.ref.table for e in r if e >= 0]
        assert self.ref.ref == [named.count(i) for i in range(len(self.ref.ref))]


@pytest.mark.parametrize("rows,table_pages,pages,page,seed", [(1, 1, 1, 8, 0), (6, 9, 30, 16, 1), (40, 33, 500, 16, 2),
                                                              (70, 130, 3000, 8, 3), (1100, 3, 2500, 64, 4),
                                                              (3, 2000, 5000, 8, 5)])
def test_a_long_run_of_calls(rows, table_pages, pages, page, seed):
    rng = random.Random(seed)
    p = Both(rows, table_pages, pages, page)
    most = table_pages * page
    length = [0] * rows
    for step in range(25):
        after = [min(most, n + rng.choice((0, 0, 1, 3, page, 2 * page + 1, rng.randint(0, most)))) for n in length]
        if p.reserve(length, after)[1] == 0:
            length = after
        p.counted()
        drop = rng.sample(range(rows), rng.randint(0, rows) // 2)
        keep = [rng.randint(0, length[r]) for r in drop]
        p.free(drop, keep)
        for r, n in zip(drop, keep):
            length[r] = n
        dst = rng.sample(range(rows), rng.randint(0, rows) // 2)
        p.free(dst, [0] * len(dst))
        for r in dst:
            length[r] = 0
        src = [r for r in range(rows) if r not in dst] or [0]
        if src != [0] or 0 not in dst:
            pick = [rng.choice(src) for _ in dst]
            part = [rng.randint(0, length[r]) for r in pick]
            p.fork(pick, dst, part)
            for d, n in zip(dst, part):
                length[d] = n
        p.counted()


def test_shared_pages_are_written_by_nobody():
    """Parent and children that all go on: each gets a copy of the page that they share."""
    p = Both(4, 4, 10)
    p.reserve([0, 0, 0, 0], [20, 0, 0, 0])
    p.fork([0, 0], [1, 2], [20, 16])
    pairs, _ = p.reserve([20, 20, 16, 0], [21, 21, 17, 0])
    assert pairs[0][0] == pairs[1][0] == 1 and pairs[0][1] != pairs[1][1] and pairs[2] == [-1, -1]
    assert p.ref.ref[1] == 0                  # nobody's any more
    p.counted()


def test_too_few_pages_change_nothing():
    p = Both(3, 6, 5)
    assert p.reserve([0, 0, 0], [40, 16, 17])[1] == 1
    assert p.reserve([0, 0, 0], [40, 16, 16])[1] == 0
    assert p.reserve([40, 16, 16], [48, 16, 18])[1] == 1
    assert p.reserve([0, 0, 0], [96, 96, 96])[1] == 13


def test_rollback_of_a_forked_row():
    """A child that goes back into shared pages without freeing them, and writes on."""
    p = Both(2, 8, 20)
    p.reserve([0, 0], [100, 0])
    p.fork([0], [1], [100])
    pairs, _ = p.reserve([100, 50], [100, 90])
    assert pairs[1][0] == p.ref.table[0][3] and len(set(p.ref.table[1][3:6]) & set(p.ref.table[0])) == 0
    p.counted()


def test_bad_calls_are_reported_and_left_out():
    p = Both(6, 4, 12)
    p.reserve([0] * 6, [40, 20, 0, 0, 0, 0])
    p.free([6, -1, 0], [0, 0, -1], error=True)
    p.fork([0, 0], [2, 2], [40, 40], error=True)          # one row twice
    p.fork([0, 2], [2, 3], [40, 0], error=True)           # a row read and written
    p.fork([0], [0], [40], error=True)
    p.fork([0], [1], [40], error=True)                    # a row that has pages
    p.fork([1, 0, 0], [2, 3, 4], [33, 65, -1], error=True)  # past the pages, past the row
    p.fork([7, 0, 0], [2, -1, 6], [0, 0, 0], error=True)
    p.fork([1, 0], [2, 3], [32, 0])
    p.reserve([-1, 20, 0, 0, 0, 0], [5, 65, 0, 0, 0, 17], error=True)
    p.reserve([2 ** 31 - 1] * 6, [-2 ** 31] * 6)
    # entries past the pool stay
    p.pool.table[5, 0] = 12
    p.ref.table[5][0] = 12
    p.free([5], [0], error=True)
    p.reserve([0] * 6, [0, 0, 0, 0, 0, 5], error=True)


def test_rows_named_twice_are_freed_once():
    p = Both(2, 6, 12)
    p.reserve([0, 0], [96, 90])
    p.pool.free(i32([0, 1, 0]), i32([50, 90, 20]))
    p.ref.free([0, 1, 0], [50, 90, 20])
    p.same()
    p.counted()


def test_a_page_that_nobody_counts_is_reported():
    p = Both(1, 2, 3)
    p.reserve([0], [32])
    p.pool.ref.zero_()
    p.ref.ref = [0] * 3
    p.free([0], [0], error=True)


def test_graph_replay_and_another_stream():
    p = Both(3, 4, 12)
    before, after = i32([0, 0, 0]), i32([20, 0, 0])
    pairs, missing = p.pool.reserve(before, after)
    p.ref.reserve([0, 0, 0], [20, 0, 0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    src, dst, n, none = i32([0]), i32([1]), i32([20]), i32([0])
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            p.pool.free(dst, none)
            p.pool.fork(src, dst, n)
            p.pool.reserve(before, after, pairs=pairs, missing=missing)
    before.copy_(i32([20, 20, 0]))
    after.copy_(i32([20, 30, 9]))
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            graph.replay()
            p.ref.free([1], [0])
            p.ref.fork([0], [1], [20])
            want = p.ref.reserve([20, 20, 0], [20, 30, 9])
    torch.cuda.synchronize()
    assert pairs.cpu().tolist() == want[0] and missing.tolist() == [0]
    p.same()
    p.counted()


def test_empty_calls():
    p = Both(2, 3, 4)
    p.free([], [])
    p.fork([], [], [])
    p.reserve([0, 0], [0, 0])
    empty = PagePool.empty(p.plan, 0, 1, 1)
    pairs, missing = empty.reserve(i32([]), i32([]))
    assert pairs.shape == (0, 2) and missing.tolist() == [0]
