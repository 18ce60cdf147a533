"""Trees, pages and sampling together, as examples/tree_decode.py uses them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from examples import tree_decode as X  # noqa: E402


def prompts(shape, n, T=37):
    return torch.randint(0, shape.vocab, (n, T), generator=torch.Generator().manual_seed(3)).tolist()


def counts_are_the_entries(model):
    table, ref = model.pool.table.cpu(), model.pool.ref.cpu()
    assert torch.equal(torch.bincount(table[table >= 0].long(), minlength=ref.numel()).int(), ref)


@pytest.mark.parametrize("samples", [1, 3])
def test_greedy_text_is_the_same_with_and_without_trees(samples):
    shape = X.Shape(dtype="f32", vocab=24)
    p = prompts(shape, 2)
    plain, rate, model = X.generate(shape, p, samples, 40, 0)
    assert rate == 1.0
    counts_are_the_entries(model)
    for branches, depth in ((1, 4), (4, 5), (9, 7)):
        text, rate, model = X.generate(shape, p, samples, 40, branches, depth)
        n = min(len(t) for t in text + plain)
        assert n >= 37 + 40 and [t[:n] for t in text] == [t[:n] for t in plain]
        assert rate > 1.05                         # some drafts are kept, or the test says nothing
        counts_are_the_entries(model)
        # greedy samples of one prompt are one text
        assert all(text[i][:n] == text[i - i % samples][:n] for i in range(len(text)))


def test_sampled_runs_are_repeatable_and_leave_no_page_behind():
    shape = X.Shape()
    p = prompts(shape, 3)
    a, _, model = X.generate(shape, p, 4, 32, 3, temperature=0.9, top_p=0.9, seed=5)
    b, _, _ = X.generate(shape, p, 4, 32, 3, temperature=0.9, top_p=0.9, seed=5)
    c, _, _ = X.generate(shape, p, 4, 32, 3, temperature=0.9, top_p=0.9, seed=6)
    assert a == b and a != c
    assert len({tuple(t) for t in a}) > 3          # the samples of a prompt part
    rows = model.pool.table.shape[0]
    model.pool.free(X.int32(list(range(rows))), X.int32([0] * rows))
    assert not model.pool.ref.any() and (model.pool.table == -1).all()
    assert model.plan.get_error()[0] == 0
