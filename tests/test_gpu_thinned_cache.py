"""Attention over sequences whose cached tokens were thinned out, on a GB300 against float64.  The kept keys
stay rotated to the positions they had, so what follows is rotated to positions of the caller's, past those: by
the norm and rotation call, and appended without a rope table."""
import random

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from hashed_gram_embedding_engram_gb300 import AttentionPlan, DraftTree, PagedCache, SequenceBatch, _lib  # noqa: E402
from oracle import decoding_oracle as O  # noqa: E402
from test_gpu_attention import U, f64  # noqa: E402
from test_gpu_pages import bits, i32  # noqa: E402

PAGE, H, HKV, D = 16, 4, 2, 64


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("parents", [[-1], [-1, 0, 0, 1, 2, 2], [-1] + [i // 2 for i in range(39)]], ids=["one", "few", "many"])
def test_what_follows_a_thinned_text(parents, dtype):
    text, kept, n = (300, 77), (140, 30), len(parents)
    plan = AttentionPlan(heads=H, heads_kv=HKV, head_dim=D, page=PAGE, dtype=dtype)
    rope, pages = plan.rope_table(512), 40
    cache = PagedCache.empty(plan, pages)
    cache.k.zero_()
    cache.v.zero_()
    table = np.array(random.Random(1).sample(range(pages), 38)).reshape(2, 19)
    g = torch.Generator(device="cuda").manual_seed(2)
    rand = lambda t, h: torch.randn(t, h, D, generator=g, device="cuda").to(plan.torch_dtype)  # noqa: E731
    start = np.array([0, text[0], sum(text)])
    whole = SequenceBatch(i32(start), i32(text), i32(table))
    cache.append(whole, rand(sum(text), HKV), rand(sum(text), HKV), rope)

    path = np.full((2, max(kept)), -1, np.int64)
    for b in range(2):
        path[b, :kept[b]] = sorted(random.Random(b).sample(range(text[b]), kept[b]))
    want = [O.compact(bits(x).cpu().numpy(), table, start, text, path, kept) for x in (cache.k, cache.v)]
    cache.compact(whole, i32(path), i32(kept))

    # the new tokens stand behind the kept ones in the cache, and behind the whole text in position
    start = np.array([0, n, 2 * n])
    length = [m + n for m in kept]
    batch = SequenceBatch(i32(start), i32(length), i32(table), max_new=n)
    tree = DraftTree(plan, batch, i32(parents * 2))
    sees, at = O.layout(parents * 2, start, length)
    assert tree.positions.cpu().tolist() == at.tolist()
    shift = i32(np.repeat(np.array(text) - np.array(kept), n))
    q, k, v = rand(2 * n, H), rand(2 * n, HKV), rand(2 * n, HKV)
    q, k = plan.qk_norm_rope(q, k, tree.positions + shift, rope)
    cache.append(batch, k, v)
    for x, w, fresh in ((cache.k, want[0], k), (cache.v, want[1], v)):
        for b in range(2):
            for i in range(n):
                slot = kept[b] + i
                w[table[b, slot // PAGE], :, slot % PAGE] = bits(fresh[b * n + i].contiguous()).cpu().numpy()
        assert (bits(x).cpu().numpy() == w).all()      # appended as they are

    out, lse = cache.attend_tree(tree, q)
    pages64 = [x.double().cpu().numpy() for x in (cache.k, cache.v)]
    scale = D ** -0.5
    ref, ref_lse, mag = O.tree_attention(f64(q), *pages64, start, length, table, scale, sees, at)
    S = scale * D * float(q.float().abs().max()) * float(cache.k.float().abs().max()) * 0.5
    L = max(length) + 1
    # as in the tests of trees: each score's products and sums, the sums of L terms, the exponentials
    bound = (2 * (D + 4) * U * S + L * U + 2.0 ** -20) * mag + 1e-30
    if dtype == "bf16":
        bound = bound + 2.0 ** -8 * np.abs(ref) + 2.0 ** -8 * mag
    assert (np.abs(f64(out) - ref) <= bound).all()
    tol = (D + 4) * U * S + L * U + 2.0 ** -20 * (1 + np.abs(ref_lse))
    assert (np.abs(f64(lse) - ref_lse) <= tol).all()
    assert plan.get_error()[0] == _lib.OK
