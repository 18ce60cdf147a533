"""Batches around the sizes at which the kernels change their ways: as many sequences as a block of
an attention kernel has threads (160, 640, 256), and the draft check's clusters of 8, 4 and 2
blocks a sequence (up to 38, up to 76, more, on 152 SMs)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from hashed_gram_embedding_engram_gb300 import SequenceBatch  # noqa: E402
from test_gpu_attention import Case, check_verify, draft_inputs  # noqa: E402


def batch_of(B, dtype, chunks, window=0):
    """B ragged sequences of 0 to 60 tokens and 0 to 2 new ones, idle and empty ones and some longer
    chunks among them; without `chunks` the launch is the one of few rows."""
    r = np.random.RandomState(B)
    new, length = r.randint(0, 3, B), r.randint(0, 61, B)
    length[r.rand(B) < 0.1] = 0
    new[0], length[B // 2], new[B - 1], length[B - 1] = 0, 300, 1, 33
    if chunks:
        new[B // 3], length[B // 3] = 90, 100
    c = Case(seed=B, dtype=dtype, heads=2, heads_kv=1, D=64, page=8, new=new.tolist(), length=length.tolist(),
             window=window)
    c.batch = SequenceBatch(c.batch.start, c.batch.length, c.batch.table, max_new=0 if chunks else 2)
    return c


@pytest.mark.parametrize("B", [159, 160, 161, 319, 320, 321, 500])
def test_attention_of_few_rows(B):
    c = batch_of(B, "bf16", False)
    c.check(*c.run())


@pytest.mark.parametrize("B", [639, 640, 641, 1281])
def test_attention_of_chunks(B):
    c = batch_of(B, "bf16", True, window=40 if B == 641 else 0)
    c.check(*c.run())


@pytest.mark.parametrize("chunks", [False, True], ids=["rows16", "rows64"])
@pytest.mark.parametrize("B", [255, 256, 257, 513, 700])
def test_attention_on_the_cuda_cores(B, chunks):
    c = batch_of(B, "f32", chunks)
    c.check(*c.run())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("B", [38, 39, 76, 77, 152, 153, 256, 400])
def test_draft_check(B, certain, dtype):
    for V in (1000, 257):
        target, draft, drafts, u = draft_inputs(B, 3, V, B, dtype, certain)
        n = torch.randint(0, 4, (B,), generator=torch.Generator().manual_seed(B), dtype=torch.int32)
        check_verify(target, draft, drafts, n, u)
