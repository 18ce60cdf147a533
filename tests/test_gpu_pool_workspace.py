"""Extending a pool's rows on a GB300 after the pool was dropped: a captured call and one that is still queued
on another stream work in memory that nothing else is given."""
import gc

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from hashed_gram_embedding_engram_gb300 import PagePool, _lib  # noqa: E402
from oracle import decoding_oracle as O  # noqa: E402
from test_gpu_pages import i32, make_plan  # noqa: E402

ROWS, PER, PAGES, PAGE = 40, 6, 300, 16
BEFORE, AFTER = [0] * ROWS, [r % (PER * PAGE) for r in range(7, 7 + 3 * ROWS, 3)]


def tensors():
    return (torch.full((ROWS, PER), -1, dtype=torch.int32, device="cuda"),
            torch.zeros(PAGES, dtype=torch.int32, device="cuda"))


def want():
    p = O.Pool([[-1] * PER] * ROWS, [0] * PAGES, PAGE)
    pairs, missing = p.reserve(BEFORE, AFTER)
    assert missing == 0
    return p, pairs


def used_by_others(size):
    """What the allocator gives next, full of numbers that are no rows and no pages."""
    return [torch.full((size,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(64)]


def same(plan, table, ref, pairs, missing):
    p, expected = want()
    torch.cuda.synchronize()
    assert table.cpu().tolist() == p.table and ref.cpu().tolist() == p.ref
    assert pairs.cpu().tolist() == expected and missing.tolist() == [0] and plan.get_error()[0] == _lib.OK


def test_a_captured_call_outlives_its_pool():
    plan = make_plan(PAGE)
    table, ref = tensors()
    before, after = i32(BEFORE), i32(AFTER)
    pool = PagePool(plan, table, ref)
    size = pool.workspace_bytes
    pool.reserve(before, before)                       # nothing, outside the graph
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pairs, missing = pool.reserve(before, after)
    del pool
    gc.collect()
    others = used_by_others(size)
    for _ in range(2):
        table.fill_(-1)
        ref.zero_()
        graph.replay()
        same(plan, table, ref, pairs, missing)
    assert all(bool((t == 0x7F).all()) for t in others)


def test_a_queued_call_on_another_stream_outlives_its_pool():
    plan = make_plan(PAGE)
    table, ref = tensors()
    before, after = i32(BEFORE), i32(AFTER)
    pool = PagePool(plan, table, ref)
    pairs, missing = i32([[0, 0]] * ROWS), i32([5])
    size = pool.workspace_bytes
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        big = torch.zeros(1 << 28, device="cuda")
        for _ in range(20):                            # some milliseconds of work before the call
            big.add_(1)
        pool.reserve(before, after, pairs=pairs, missing=missing)
    del pool
    gc.collect()
    others = used_by_others(size)
    same(plan, table, ref, pairs, missing)
    assert all(bool((t == 0x7F).all()) for t in others)
