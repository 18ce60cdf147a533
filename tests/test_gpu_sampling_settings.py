"""Settings at the ends of their types on a GB300, where several blocks share a row: tokens equal to those of
whole numbers in Python, and to those of the setting that is off."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from hashed_gram_embedding_engram_gb300 import sample_tokens  # noqa: E402
from test_gpu_sampling import check, normal  # noqa: E402


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [9000, 129280, 600001])
def test_top_k_of_any_size_in_rows_of_several_blocks(V, dtype):
    logits, u = normal(4, V, 21, dtype=dtype)
    top = torch.tensor([2 ** 31 - 1, 2 ** 31 - 8, -2 ** 31, V], dtype=torch.int32, device="cuda")
    for settings in (dict(), dict(top_p=0.9), dict(temperature=0.0), dict(min_p=0.02)):
        off = sample_tokens(logits, u, **settings)
        for k in (top, 2 ** 31 - 1, 10 ** 30, -(10 ** 30)):
            assert torch.equal(sample_tokens(logits, u, top_k=k, **settings), off)
    check(logits, u, top_k=top, top_p=0.9)
