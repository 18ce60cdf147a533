"""Forks whose rows meet, on a GB300: of a chain of pairs those are left out whose dst another pair reads or
writes, and the others are made."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from test_gpu_pages import Both  # noqa: E402


@pytest.mark.parametrize("src,dst,made", [([0, 1], [1, 2], {2: 1}),                 # 1 is read: it is not written
                                          ([1, 0], [2, 1], {2: 1}),
                                          ([0, 3, 1], [3, 2, 4], {4: 1}),           # 3 has no pages
                                          ([0, 1, 0], [2, 3, 3], {2: 0}),           # 3 is named twice
                                          ([0, 1, 0, 1], [2, 3, 4, 0], {2: 0, 3: 1, 4: 0}),
                                          ([0, 0, 0, 1], [2, 3, 4, 5], {2: 0, 3: 0, 4: 0, 5: 1})])
def test_pairs_that_read_another_pairs_dst_are_made(src, dst, made):
    p = Both(6, 4, 30)
    p.reserve([0] * 6, [40, 33, 0, 0, 0, 0])
    rows = [list(r) for r in p.ref.table]
    length = [33 if a in (0, 1) else 20 for a in src]
    p.fork(src, dst, length, error=len(made) < len(src))
    for d in range(2, 6):
        assert p.ref.table[d] == (rows[made[d]][:3] + [-1] if d in made else [-1] * 4)
    assert p.ref.table[:2] == rows[:2]
    p.counted()


def test_many_pairs_that_meet():
    """More pairs than a block has threads; every third dst is another pair's src."""
    n = 400
    p = Both(3 * n, 3, 4 * n)
    p.reserve([0] * (3 * n), [20] * n + [0] * (2 * n))
    src, dst = list(range(n)), [n + i if i % 3 else (i + 1) % n for i in range(n)]
    p.fork(src, dst, [17] * n, error=True)
    made = [i for i in range(n) if i % 3]
    assert [r for r in range(n, 3 * n) if p.ref.table[r][0] >= 0] == [n + i for i in made]
    assert all(p.ref.table[n + i] == p.ref.table[i] for i in made)
    p.counted()
