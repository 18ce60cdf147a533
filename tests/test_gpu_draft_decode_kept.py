"""The draft loop where drafts are kept: prompts that repeat their n-grams."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from examples import draft_decode as E  # noqa: E402


def test_kept_and_turned_down_drafts_leave_the_greedy_text(monkeypatch):
    """Steps that keep none, some and all of their drafts, and the text of single-token steps: the
    states and caches are those of the kept tokens."""
    seen, check = [], E.verify_drafts

    def verify(p, drafts, u, n_drafts=None):
        tokens, accepted = check(p, drafts, u, n_drafts=n_drafts)
        seen.extend(zip(n_drafts.tolist(), accepted.tolist()))
        return tokens, accepted

    monkeypatch.setattr(E, "verify_drafts", verify)
    shape = E.Shape(dtype="f32")
    prompts = torch.randint(0, shape.vocab, (3, 8), generator=torch.Generator().manual_seed(1)).repeat(1, 5)
    plain, _ = E.generate(shape, prompts, 96, 0, greedy=True)
    seen.clear()
    text, rate = E.generate(shape, prompts, 96, 4, greedy=True)
    assert rate > 1.0 and all(0 <= a <= n for n, a in seen)
    assert any(a == 0 < n for n, a in seen) and any(0 < a < n for n, a in seen) and any(0 < a == n for n, a in seen)
    for a, b in zip(text, plain):
        n = min(len(a), len(b))
        assert n >= 40 + 60 and a[:n] == b[:n]
