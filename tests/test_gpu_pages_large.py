"""Sizes at which the page operators take further rounds, on a GB300 against plain Python: paths of more rows
than a block looks up at once (8192), tables of more rows than shared memory has places for (2048), pools whose
unused pages lie past the first 8192; bad paths and pages among long paths.  Everything has to be equal."""
import random
from collections import Counter

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from hashed_gram_embedding_engram_gb300 import SequenceBatch, _lib  # noqa: E402
from oracle import decoding_oracle as O  # noqa: E402
from test_gpu_pages import Both, bits, i32, make_plan, random_cache  # noqa: E402


# ---------------------------------------------------------------- rows moved together
def paths(seed, new, count, width=None):
    """Ascending paths, the first rows in place already."""
    rng = random.Random(seed)
    path = np.full((len(new), width or max(count)), 123456, np.int64)
    for b, (n, c) in enumerate(zip(new, count)):
        stay = min(5, c)
        path[b, :c] = list(range(stay)) + sorted(rng.sample(range(stay, n), c - stay))
    return path


def tables(seed, length, page):
    """(table, pages) with the sequences' pages in any order and two of nobody."""
    used = [-(-m // page) for m in length]
    order = list(range(sum(used) + 2))
    random.Random(seed).shuffle(order)
    table, at = np.full((len(length), max(used)), -1, np.int64), 0
    for b, m in enumerate(used):
        table[b, :m] = order[at:at + m]
        at += m
    return table, len(order)


def moved(cache, plan, table, new, length, path, count, status):
    start = np.concatenate(([0], np.cumsum(new)))
    want = [O.compact(bits(x).cpu().numpy(), table, start, length, path, count) for x in (cache.k, cache.v)]
    cache.compact(SequenceBatch(i32(start), i32(length), i32(table)), i32(path), i32(count))
    for x, w in zip((cache.k, cache.v), want):
        assert (bits(x).cpu().numpy() == w).all()
    assert plan.get_error()[0] == status


@pytest.mark.parametrize("dtype,page,heads_kv,D", [("bf16", 8, 2, 64), ("f32", 64, 1, 96), ("bf16", 1024, 1, 128),
                                                   ("bf16", 16, 3, 8)])
@pytest.mark.parametrize("count", [8191, 8192, 8193, 16384, 16385, 20000])
def test_paths_of_several_rounds(count, dtype, page, heads_kv, D):
    """With text before them that does not end with a page, so that every round begins inside one."""
    new, length = [count + 1500], [count + 1500 + 13]
    table, pages = tables(count, length, page)
    plan = make_plan(page, dtype, heads_kv, D)
    moved(random_cache(plan, pages, count), plan, table, new, length, paths(count, new, [count]), [count], _lib.OK)


def test_sequences_of_one_round_and_of_several():
    new, count = [9000, 40, 20000, 8200], [8500, 0, 17000, 8200]
    length = [n + m for n, m in zip(new, (0, 3, 77, 16))]
    table, pages = tables(1, length, 16)
    plan = make_plan(16, "bf16", 2, 64)
    moved(random_cache(plan, pages), plan, table, new, length, paths(2, new, count), count, _lib.OK)


def test_long_paths_that_do_not_ascend_move_nothing():
    new, length, n = [9000, 500], [9100, 533], 8700
    table, pages = tables(3, length, 16)
    plan = make_plan()
    good = paths(4, new, [n, 300], n + 40)
    for at, value in ((0, -1), (1, 0), (40, 39), (300, 12345), (8191, 5), (8192, 8191), (n - 1, 9000), (n - 1, -2 ** 31)):
        path = good.copy()
        path[0, at] = value
        if at == 8192:
            path[0, at] = path[0, at - 1]             # the same row again, where a round begins
        moved(random_cache(plan, pages, at), plan, table, new, length, path, [n, 300], _lib.ERR_INDEX_RANGE)
    for count in (-1, n + 41, 2 ** 31 - 1, -2 ** 31):
        moved(random_cache(plan, pages, 9), plan, table, new, length, good, [count, 300], _lib.ERR_INDEX_RANGE)
    # more rows than the sequence has new tokens; a sequence whose length is below them
    moved(random_cache(plan, pages, 10), plan, table, [500, 500], length, good, [n, 300], _lib.ERR_INDEX_RANGE)
    moved(random_cache(plan, pages, 11), plan, table, new, [8999, 533], good, [n, 300], _lib.ERR_INDEX_RANGE)
    moved(random_cache(plan, pages, 12), plan, table, new, length, good, [0, 300], _lib.OK)


@pytest.mark.parametrize("entry", [-1, -2 ** 31, 10 ** 6, 2 ** 31 - 1])
@pytest.mark.parametrize("at", [0, 3, 260, 513, 560])
def test_bad_pages_are_left_out_of_a_long_move(at, entry):
    """Pages that rows come from, go to, or both; in the first round and in the second."""
    new, length, count = [9000], [9010], 8700
    table, pages = tables(5, length, 16)
    table[0, at] = entry
    plan = make_plan()
    moved(random_cache(plan, pages), plan, table, new, length, paths(6, new, [count]), [count], _lib.ERR_INDEX_RANGE)


# ---------------------------------------------------------------- the table
def counted(p):
    named = Counter(e for r in p.ref.table for e in r if e >= 0)
    assert p.ref.ref == [named[i] for i in range(len(p.ref.ref))]


@pytest.mark.parametrize("rows,table_pages,pages", [(2047, 2, 5000), (2048, 3, 7000), (2049, 3, 7000), (5000, 2, 12000)])
def test_tables_of_many_rows(rows, table_pages, pages):
    rng, p = random.Random(rows), Both(rows, table_pages, pages)
    most, length = 16 * table_pages, [0] * rows
    for step in range(4):
        after = [min(most, n + rng.choice((0, 0, 1, 5, 16, 20))) for n in length]
        if p.reserve(length, after)[1] == 0:
            length = after
        drop = rng.sample(range(rows), rows // 3)
        p.free(drop, [0] * len(drop))
        for r in drop:
            length[r] = 0
        src = [r for r in range(rows) if length[r]]
        pick = [rng.choice(src) for _ in drop]
        p.fork(pick, drop, [length[r] for r in pick])
        for r, a in zip(drop, pick):
            length[r] = length[a]
        counted(p)
    p.reserve([0] * rows, [most] * rows)              # whole rows: new pages and copies
    counted(p)


@pytest.mark.parametrize("pages", [8192, 8193, 16384, 16385, 40500])
def test_unused_pages_past_the_first_round(pages):
    """The pool's first pages are taken, all or nearly, and rows are extended from the last ones."""
    rng, rows, per = random.Random(pages), 45, 1000
    p = Both(rows, per, pages)
    full = min(pages // per, rows - 5)
    most = [16 * per] * full + [0] * (rows - full)
    p.reserve([0] * rows, most)
    rest = pages - full * per                         # unused, the last ones
    assert all(x == 1 for x in p.ref.ref[:full * per]) and not any(p.ref.ref[full * per:])
    length = list(most)
    for step in range(3):
        after = [min(16 * per, n + rng.randint(0, 16 * rest // 30)) if r >= full else n for r, n in enumerate(length)]
        if p.reserve(length, after)[1] == 0:
            length = after
        # holes at the front, fewer than the next call asks for
        p.free([0, 1], [16 * (per - 3), 16 * (per - 1)])
        length[0], length[1] = 16 * (per - 3), 16 * (per - 1)
        counted(p)
    # copy on write where the copies lie past the first round
    children = [r for r in range(full, rows) if length[r] == 0] or [rows - 1]
    p.free(children, [0] * len(children))
    p.fork([2] * len(children), children, [16 * 7 + 5] * len(children))
    for r in children:
        length[r] = 16 * 7 + 5
    p.reserve(length, [n + 1 if r in children else n for r, n in enumerate(length)])
    counted(p)
    unused = sum(x == 0 for x in p.ref.ref)
    have = sum(e < 0 for r in p.ref.table for e in r)
    missing = p.reserve([0] * rows, [16 * per] * rows)[1]
    assert have <= unused or missing >= have - unused > 0
    counted(p)
