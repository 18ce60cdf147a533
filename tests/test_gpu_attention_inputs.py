"""Inputs of the attention sub-block that are out of range or oddly placed: what a call leaves
out, and what it takes."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from hashed_gram_embedding_engram_gb300 import _lib, verify_drafts  # noqa: E402
from oracle import attention_oracle as O  # noqa: E402
from test_gpu_attention import Case, draft_inputs  # noqa: E402

# one set of sequences for each attention kernel: few rows, chunks, and both of the CUDA cores'
KERNELS = [dict(new=(1, 2, 1), length=(200, 40, 77), heads=8, heads_kv=2, D=128),
           dict(new=(140, 2, 40), length=(200, 40, 77), heads=8, heads_kv=2, D=128),
           dict(new=(1, 2, 1), length=(200, 40, 77), dtype="f32"),
           dict(new=(140, 2, 40), length=(200, 40, 77), dtype="f32", window=50)]


@pytest.mark.parametrize("shape", KERNELS, ids=["rows", "tiles", "simt16", "simt64"])
@pytest.mark.parametrize("bad", [10 ** 9, "room + 1", -1, -2 ** 31, 2 ** 31 - 1])
@pytest.mark.parametrize("b", [0, 1, 2])
def test_queries_of_a_sequence_with_a_bad_length_see_no_key(shape, bad, b):
    """The entries of the table past a sequence's pages hold 0, as in a zero-filled table: a valid
    page, of which nothing may reach the output."""
    c = Case(seed=31, **shape)
    c.batch.table.clamp_(min=0)
    c.batch.length[b] = c.table.shape[1] * c.page + 1 if isinstance(bad, str) else bad
    out, lse = c.run()
    assert c.plan.get_error()[0] == _lib.ERR_INDEX_RANGE
    c.length[b] = 0
    c.check(out, lse)


@pytest.mark.parametrize("shape", KERNELS, ids=["rows", "tiles", "simt16", "simt64"])
def test_queries_of_a_sequence_with_a_bad_start_see_no_key(shape):
    c = Case(seed=32, **shape)
    c.batch.table.clamp_(min=0)
    n0, n1, n2 = shape["new"]
    T, length, good = n0 + n1 + n2, list(c.length), list(c.start)
    for starts, rows, lost in (([0, n0, n0 + n1, T + 1], good, (2,)), ([0, n0, n0 + n1, 2 ** 31 - 1], good, (2,)),
                               ([-3, n0, n0 + n1, T], good, (0,)), ([0, T + 900, T, T], [0, T, T, T], (0, 1))):
        c.batch.start.copy_(torch.tensor(starts, dtype=torch.int32))
        out, lse = c.run()
        assert c.plan.get_error()[0] == _lib.ERR_INDEX_RANGE
        c.start = np.array(rows, np.int32)
        c.length = [0 if b in lost else m for b, m in enumerate(length)]
        c.check(out, lse)


@pytest.mark.parametrize("what", ["length", "start"])
def test_append_and_attention_leave_out_the_same_sequences(what):
    c = Case(seed=33, new=(2, 3, 2), length=(20, 30, 33), heads=4, heads_kv=2, D=64, stale=0.0)
    c.batch.table.clamp_(min=0)
    if what == "length":
        c.batch.length[1] = 10 ** 6
    else:
        c.batch.start[0] = -2
    b = 1 if what == "length" else 0
    k = torch.full((7, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    before = c.cache.k.clone()
    c.cache.append(c.batch, k, k)
    changed = (c.cache.k != before).any(-1).any(1).nonzero().tolist()
    want = [[int(c.table[x, j // c.page]), j % c.page] for x in range(3) if x != b
            for j in range(c.length[x] - c.new[x], c.length[x])]
    assert sorted(changed) == sorted(want)
    _, lse = c.run()
    dropped = torch.zeros(7, dtype=torch.bool)
    dropped[c.start[b]:c.start[b + 1]] = True
    assert torch.equal(torch.isneginf(lse).all(1).cpu(), dropped)
    assert c.plan.get_error()[0] == _lib.ERR_INDEX_RANGE


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [257, 1000, 1001])
def test_draft_check_of_a_slice_of_a_batch(V, dtype):
    """Probabilities that begin anywhere, as those of some sequences of a batch do where a row is
    not a multiple of 16 bytes."""
    target, draft, drafts, u = draft_inputs(6, 2, V, 3, dtype)
    t, d = target.cuda(), draft.cuda()
    for b in range(6):
        x = slice(b, b + 1)
        want = O.verify(target[x].float().numpy(), draft[x].float().numpy(), drafts[x].numpy(), None, u[x].numpy())
        for draft_at in (d[x], d[x].clone()):
            tokens, accepted = verify_drafts(t[x], drafts[x].cuda(), u[x].cuda(), draft_probs=draft_at)
            assert np.array_equal(tokens.cpu().numpy(), want[0]) and np.array_equal(accepted.cpu().numpy(), want[1])
        # moved by one element from an aligned place, rows that are a multiple of 16 bytes among them
        flat = torch.empty(target[x].numel() + 1, dtype=dtype, device="cuda")
        off = flat[1:].view_as(target[x])
        off.copy_(t[x])
        tokens, accepted = verify_drafts(off, drafts[x].cuda(), u[x].cuda(), draft_probs=d[x])
        assert np.array_equal(tokens.cpu().numpy(), want[0]) and np.array_equal(accepted.cpu().numpy(), want[1])
