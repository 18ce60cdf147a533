"""The front end of trees, pages and sampling without a GPU: tensors that say they are on a GPU, and a
stand-in for the library that keeps what it is called with."""
import ctypes
import struct

import pytest
import torch

from hashed_gram_embedding_engram_gb300 import attention as A, decoding as Dm
from test_attention_front_end import B, D, F32, H, HKV, I32, OnGpu, PAGE, T, batch, cache, lib, moved, on, plan  # noqa: F401

W, ROWS, PER, PAGES, V = 4, 3, 5, 12, 50


def tree(p=None, **kw):
    return Dm.DraftTree(p or plan(), batch(), on(0, T, dtype=I32), **{"max_nodes": 32, "mask": on(0, T, 1, dtype=I32),
                                                                     "positions": on(0, T, dtype=I32), **kw})


def pool(p=None):
    x = Dm.PagePool.__new__(Dm.PagePool)
    x.plan, x.table, x.ref = p or plan(), on(0, ROWS, PER, dtype=I32), on(0, PAGES, dtype=I32)
    x._packed, x.workspace_bytes, x._workspace = b"", 64, on(0, 64, dtype=torch.uint8)
    return x


def i32(*shape):
    return on(0, *shape, dtype=I32)


CALLS = {
    "engram_tree_build": (lambda **k: Dm.DraftTree(plan(), **k),
                          lambda: dict(batch=batch(), parent=i32(T), mask=i32(T, 2), positions=i32(T))),
    "engram_tree_attention": (lambda **k: cache(plan()).attend_tree(tree(), **k),
                              lambda: dict(q=on(0, T, H, D), out=on(0, T, H, D), lse=on(0, T, H, dtype=F32),
                                           workspace=on(0, 1 << 16, dtype=torch.uint8))),
    "engram_tree_accept": (lambda **k: tree().accept(width=W, **k),
                           lambda: dict(tokens=i32(T), sampled=i32(T), path=i32(B, W), count=i32(B), emitted=i32(B, W),
                                        length=i32(B))),
    "engram_kv_compact": (lambda **k: cache(plan()).compact(**k), lambda: dict(batch=batch(), path=i32(B, W), count=i32(B))),
    "engram_kv_copy_pages": (lambda **k: cache(plan()).copy_pages(**k), lambda: dict(pairs=i32(6, 2))),
    "engram_pool_free": (lambda **k: pool().free(**k), lambda: dict(rows=i32(2), keep=i32(2))),
    "engram_pool_fork": (lambda **k: pool().fork(**k), lambda: dict(src=i32(2), dst=i32(2), length=i32(2))),
    "engram_pool_reserve": (lambda **k: pool().reserve(**k),
                            lambda: dict(before=i32(ROWS), after=i32(ROWS), pairs=i32(ROWS, 2), missing=i32(1))),
    "engram_sample_tokens": (lambda **k: Dm.sample_tokens(**k),
                             lambda: dict(logits=on(0, 3, V, dtype=F32), u=on(0, 3, dtype=F32),
                                          temperature=on(0, 3, dtype=F32), top_k=i32(3), top_p=on(0, 3, dtype=F32),
                                          min_p=on(0, 3, dtype=F32), tokens=i32(3))),
}
NAMES = [(n, k) for n, (_, args) in CALLS.items() for k in args()]


def count(lib, name):  # noqa: F811
    return [n for n, _ in lib.calls].count(name)


@pytest.mark.parametrize("name,arg", NAMES)
def test_tensors_of_another_device_are_refused(lib, name, arg):  # noqa: F811
    call, args = CALLS[name]
    call(**args())
    assert count(lib, name) == 1
    x = args()
    x[arg] = moved(x[arg])
    with pytest.raises(ValueError, match="cuda:1"):
        call(**x)
    assert count(lib, name) == 1


@pytest.mark.parametrize("name,arg", [(n, k) for n, k in NAMES if k not in ("batch", "workspace")])
def test_other_types_and_shapes_are_refused(lib, name, arg):  # noqa: F811
    call, args = CALLS[name]
    for wrong in (on(0, *args()[arg].shape, dtype=torch.float16), on(0, 7, 7, 7, dtype=args()[arg].dtype), None, 3.5):
        if wrong is None and arg in ("mask", "positions", "out", "lse", "path", "count", "emitted", "length", "pairs",
                                     "missing", "tokens", "top_k", "temperature", "top_p", "min_p"):
            continue
        if isinstance(wrong, float) and name == "engram_sample_tokens" and arg in ("temperature", "top_p", "min_p", "top_k"):
            continue
        x = args()
        x[arg] = wrong
        with pytest.raises((TypeError, ValueError, AttributeError)):
            call(**x)
    assert count(lib, name) == 0


@pytest.mark.parametrize("arg", ["logits", "u", "temperature", "top_p", "min_p"])
def test_sampling_refuses_inputs_that_require_a_gradient(lib, arg):  # noqa: F811
    call, args = CALLS["engram_sample_tokens"]
    x = args()
    x[arg].requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        call(**x)
    with torch.no_grad():
        call(**x)
    assert count(lib, "engram_sample_tokens") == 1


def test_attention_of_a_tree_refuses_queries_that_require_a_gradient(lib):  # noqa: F811
    call, args = CALLS["engram_tree_attention"]
    x = args()
    x["q"].requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        call(**x)
    with torch.no_grad():
        call(**x)


@pytest.mark.parametrize("nodes,words", [(1, 1), (32, 1), (33, 2), (64, 2), (255, 8), (256, 8)])
def test_masks_have_a_bit_for_each_node(lib, nodes, words):  # noqa: F811
    tree(max_nodes=nodes, mask=i32(T, words), window=2 ** 40)
    at = next(at for name, at in lib.calls if name == "engram_tree_build")
    assert struct.unpack("@PPii", at[3])[2:] == (words, 2 ** 31 - 1)


def test_trees_refuse_bad_sizes(lib):  # noqa: F811
    for bad in (0, -1, 257, 10 ** 9):
        with pytest.raises(ValueError, match="max_nodes"):
            tree(max_nodes=bad)
    with pytest.raises(ValueError, match="window"):
        tree(window=-1)
    t = tree()
    for bad in (0, -3, 257):
        with pytest.raises(ValueError, match="width"):
            t.accept(i32(T), i32(T), width=bad)
    with pytest.raises(ValueError, match="shape"):       # queries of another number of tokens than the tree's
        cache(plan()).attend_tree(t, on(0, T + 1, H, D))
    other = plan()
    other.device = 1
    t.plan = other
    with pytest.raises(ValueError, match="cuda:0"):
        cache(plan()).attend_tree(t, on(0, T, H, D))


@pytest.mark.parametrize("call", ["build", "accept", "attend_tree", "compact", "copy_pages", "free", "fork", "reserve"])
def test_calls_of_a_closed_plan_are_refused(lib, call):  # noqa: F811
    p = plan()
    c, t, q = cache(p), tree(p), pool(p)
    p.close()
    n = len(lib.calls)
    with pytest.raises(ValueError, match="closed"):
        {"build": lambda: tree(p), "accept": lambda: t.accept(i32(T), i32(T)), "attend_tree": lambda: c.attend_tree(t, on(0, T, H, D)),
         "compact": lambda: c.compact(batch(), i32(B, W), i32(B)), "copy_pages": lambda: c.copy_pages(i32(2, 2)),
         "free": lambda: q.free(i32(1), i32(1)), "fork": lambda: q.fork(i32(1), i32(1), i32(1)),
         "reserve": lambda: q.reserve(i32(ROWS), i32(ROWS))}[call]()
    assert len(lib.calls) == n


def test_settings_reach_the_library_as_numbers_or_tensors(lib):  # noqa: F811
    call, args = CALLS["engram_sample_tokens"]
    x = args()
    call(logits=x["logits"], u=x["u"], temperature=0.5, top_k=2 ** 40, top_p=x["top_p"], tokens=x["tokens"])
    got = struct.unpack("@PPPPfiff", lib.calls[-1][1][4])
    assert got[:4] == (0, 0, x["top_p"].data_ptr(), 0) and got[4:] == (0.5, 2 ** 31 - 1, 0.0, 0.0)
    call(logits=x["logits"], u=x["u"], top_k=-7, tokens=x["tokens"])
    assert struct.unpack("@PPPPfiff", lib.calls[-1][1][4])[4:] == (1.0, -1, 1.0, 0.0)


def test_logits_have_dense_rows_that_do_not_overlap(lib):  # noqa: F811
    x = on(0, 3, 2 * V, dtype=F32)
    u, out = on(0, 3, dtype=F32), i32(3)
    Dm.sample_tokens(x[:, :V], u, tokens=out)
    assert lib.calls[-1][1][2] == 2 * V and lib.calls[-1][1][5:7] == (3, V)
    for bad in (x[:, ::2], x.T, x[:, :V].as_strided((3, V), (V - 1, 1)).as_subclass(OnGpu), x[:1, :V].expand(3, V)):
        with pytest.raises(ValueError):
            Dm.sample_tokens(bad, on(0, bad.shape[0], dtype=F32), tokens=i32(bad.shape[0]))
    Dm.sample_tokens(x[:1, :V].as_strided((1, V), (0, 1)).as_subclass(OnGpu), u[:1], tokens=out[:1])
    assert lib.calls[-1][1][2] == V


def test_sampling_runs_on_the_current_device(lib, monkeypatch):  # noqa: F811
    call, args = CALLS["engram_sample_tokens"]
    everything = {k: moved(v) for k, v in args().items()}
    with pytest.raises(ValueError, match="cuda:1"):
        call(**everything)
    monkeypatch.setattr(A, "_current_device", lambda: 1)
    call(**everything)


def test_a_pool_is_packed_as_the_header_says(lib, monkeypatch):  # noqa: F811
    table, ref = i32(ROWS, PER), i32(PAGES)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: on(0, 8, dtype=torch.uint8))
    p = Dm.PagePool(plan(), table, ref)
    assert struct.unpack("@PPiiq", p._packed) == (table.data_ptr(), ref.data_ptr(), ROWS, PER, PAGES)
    for bad in ((ref, ref), (table, table), (table.float(), ref), (moved(table), ref), (table, moved(ref))):
        with pytest.raises((TypeError, ValueError)):
            Dm.PagePool(plan(), *bad)
    assert isinstance(p.plan._h, ctypes.c_void_p)
