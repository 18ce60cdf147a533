"""Where the memory lies that extending a pool's rows works in, without a GPU: it belongs to the call's stream, or
to the graph that the call is captured in, so that neither a pool that is dropped nor another stream's call
takes it from what is still queued."""
import pytest
import torch

from hashed_gram_embedding_engram_gb300 import attention as A
from test_attention_front_end import lib  # noqa: F401
from test_decoding_front_end import ROWS, i32, pool


@pytest.fixture
def reserve(lib, monkeypatch):  # noqa: F811
    """reserve(pool, stream, capturing): where the call's memory lies, and whether it was allocated by it."""
    made, empty = [], torch.empty

    def kept_empty(*shape, **options):
        made.append(empty(*shape, **options))
        return made[-1]

    def call(p, stream, capturing=False):
        n = len(made)
        monkeypatch.setattr(A, "_current_stream", lambda device: stream)
        monkeypatch.setattr(A, "_capturing", lambda: capturing)
        p.reserve(i32(ROWS), i32(ROWS), pairs=i32(ROWS, 2), missing=i32(1))
        name, args = lib.calls[-1]
        assert name == "engram_pool_reserve" and args[8] == stream and args[7] == p.workspace_bytes
        assert [t.numel() >= args[7] for t in made if t.data_ptr() == args[6]] == [True]
        return args[6], any(t.data_ptr() == args[6] for t in made[n:])

    monkeypatch.setattr(torch, "empty", kept_empty)
    return call


def test_each_stream_has_memory_of_its_own(reserve):
    p = pool()
    first = {s: reserve(p, s) for s in (0, 7, 9)}
    assert len({at for at, _ in first.values()}) == 3 and all(new for _, new in first.values())
    for s in (9, 0, 7, 0):                            # allocated once, while the stream was current
        assert reserve(p, s) == (first[s][0], False)
    assert reserve(pool(), 7)[1]                      # of each pool


def test_each_captured_call_has_memory_of_its_own(reserve):
    p = pool()
    at = [reserve(p, 7)[0]] + [reserve(p, 7, capturing=True)[0] for _ in range(3)]
    assert len(set(at)) == 4
    assert reserve(p, 7) == (at[0], False) and reserve(p, 7, capturing=True)[1]
