"""The n-gram draft loop of examples/draft_decode.py: Engram layer, paged cache, attention and
draft check together."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from examples.draft_decode import Shape, generate  # noqa: E402


def prompts(vocab, B=3, T=40):
    return torch.randint(0, vocab, (B, T), generator=torch.Generator().manual_seed(1))


def test_greedy_text_does_not_depend_on_drafts():
    """With a target that puts all weight on its best token, a draft is kept exactly if it is that
    token: the text is the one of single-token steps.  fp32, where the chunked and the single-token
    pass differ by rounding only (about 1e-6, against gaps of 1e-3 and more between the best two)."""
    shape = Shape(dtype="f32")
    plain, rate0 = generate(shape, prompts(shape.vocab), 48, 0, greedy=True)
    assert rate0 == 1.0
    for S in (1, 4):
        text, rate = generate(shape, prompts(shape.vocab), 48, S, greedy=True)
        for a, b in zip(text, plain):
            n = min(len(a), len(b))
            assert n >= 40 + 20 and a[:n] == b[:n]
        assert 1.0 <= rate <= S + 1


def test_sampled_text_is_in_the_vocabulary():
    shape = Shape(dtype="bf16")
    text, rate = generate(shape, prompts(shape.vocab), 24, 3, greedy=False)
    assert all(0 <= t < shape.vocab for x in text for t in x) and 1.0 <= rate <= 4.0
