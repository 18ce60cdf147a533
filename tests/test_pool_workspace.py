"""Where the memory lies that extending a pool's rows works in, without a GPU: it belongs to the call, so
that neither a pool that is dropped nor another stream's call takes it from what is still queued."""
import torch

from test_attention_front_end import lib  # noqa: F401
from test_decoding_front_end import ROWS, count, i32, pool


def test_each_reserve_has_memory_of_its_own(lib, monkeypatch):  # noqa: F811
    made, empty = [], torch.empty

    def kept_empty(*shape, **options):
        made.append(empty(*shape, **options))
        return made[-1]

    p = pool()
    monkeypatch.setattr(torch, "empty", kept_empty)
    for _ in range(3):
        p.reserve(i32(ROWS), i32(ROWS), pairs=i32(ROWS, 2), missing=i32(1))
    assert count(lib, "engram_pool_reserve") == 3
    used = [args[6:8] for name, args in lib.calls if name == "engram_pool_reserve"]
    assert len({at for at, _ in used}) == 3
    for at, size in used:
        assert [t.numel() >= size == p.workspace_bytes for t in made if t.data_ptr() == at] == [True]
