"""Arguments of trees, pages and sampling that are no tensors, or tensors of another rank, without a GPU: refused by
name, as TypeError or ValueError, before the library is called."""
import pytest
import torch

from hashed_gram_embedding_engram_gb300 import decoding as Dm
from test_attention_front_end import D, F32, H, I32, T, cache, lib, on, plan  # noqa: F401
from test_decoding_front_end import V, count, i32, pool, tree

NONE = (0.5, [0], None, "x")
RANKS = (i32(), i32(2, 1))
CALLS = {
    "engram_pool_free": (lambda **k: pool().free(**k), lambda: dict(rows=i32(2), keep=i32(2))),
    "engram_pool_fork": (lambda **k: pool().fork(**k), lambda: dict(src=i32(2), dst=i32(2), length=i32(2))),
}


@pytest.mark.parametrize("name,arg", [(n, k) for n, (_, args) in CALLS.items() for k in args()])
def test_rows_that_are_no_rows(lib, name, arg):  # noqa: F811
    call, args = CALLS[name]
    for wrong in (*NONE, *RANKS):
        with pytest.raises((TypeError, ValueError), match=f"^{arg}: "):
            call(**{**args(), arg: wrong})
    assert count(lib, name) == 0


@pytest.mark.parametrize("grad", [True, False])
def test_random_numbers_that_are_no_tensor(lib, grad):  # noqa: F811
    for wrong in NONE:
        with torch.set_grad_enabled(grad), pytest.raises((TypeError, ValueError), match="^u: "):
            Dm.sample_tokens(on(0, 3, V, dtype=F32), wrong, tokens=i32(3))
    assert count(lib, "engram_sample_tokens") == 0


@pytest.mark.parametrize("name", ["temperature", "top_k", "top_p", "min_p"])
def test_settings_that_are_no_numbers(lib, name):  # noqa: F811
    for wrong in (None, "x", [0.5], (1, 2)):
        with pytest.raises((TypeError, ValueError), match=f"^{name}: "):
            Dm.sample_tokens(on(0, 3, V, dtype=F32), on(0, 3, dtype=F32), tokens=i32(3), **{name: wrong})
    assert count(lib, "engram_sample_tokens") == 0


@pytest.mark.parametrize("grad", [True, False])
def test_queries_that_are_no_queries(lib, grad):  # noqa: F811
    for wrong in (*NONE, on(0), on(0, T, H), on(0, T + 1, H, D), on(0, T, H, D, dtype=I32)):
        with torch.set_grad_enabled(grad), pytest.raises((TypeError, ValueError), match="^q: "):
            cache(plan()).attend_tree(tree(), wrong)
    assert count(lib, "engram_tree_attention") == 0


def test_more_rows_than_a_call_takes(lib):  # noqa: F811
    n = 65536
    for call in (lambda n: pool().free(i32(n), i32(n)), lambda n: pool().fork(i32(n), i32(n), i32(n))):
        call(n)
        with pytest.raises(ValueError, match="65536"):
            call(n + 1)
    assert (count(lib, "engram_pool_free"), count(lib, "engram_pool_fork")) == (1, 1)
    for rows in (n, n + 1):
        p = pool()
        p.table = i32(rows, 2)
        outputs = dict(pairs=i32(rows, 2), missing=i32(1))
        if rows == n:
            p.reserve(i32(rows), i32(rows), **outputs)
        else:
            with pytest.raises(ValueError, match="^table: 65537 rows"):
                p.reserve(i32(rows), i32(rows), **outputs)
    assert count(lib, "engram_pool_reserve") == 1
