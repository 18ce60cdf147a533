"""The attention sub-block's front end without a GPU: tensors that say they are on a GPU, and a
stand-in for the library that keeps what it is called with."""
import ctypes

import pytest
import torch

from hashed_gram_embedding_engram_gb300 import _lib, attention as A


class OnGpu(torch.Tensor):
    """A host tensor that calls itself one of GPU `device`."""
    is_cuda = True
    index = 0

    def get_device(self):
        return self.index


def on(device, *shape, dtype=torch.bfloat16):
    t = torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)
    t.index = device
    return t


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    x = Library()
    monkeypatch.setattr(_lib, "_lib", lambda: x)
    monkeypatch.setattr(A, "_current_stream", lambda device: 0)
    monkeypatch.setattr(A, "_current_device", lambda: 0)
    monkeypatch.setattr(A, "_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return x


T, H, HKV, D, PAGE, B = 4, 4, 2, 64, 16, 2
I32, F32 = torch.int32, torch.float32


def plan():
    p = A.AttentionPlan(heads=H, heads_kv=HKV, head_dim=D, page=PAGE)
    p.workspace_bytes = 1 << 16
    p._h = ctypes.c_void_p(1)
    return p


def batch(device=0):
    return A.SequenceBatch(on(device, B + 1, dtype=I32), on(device, B, dtype=I32), on(device, B, 3, dtype=I32), max_new=2)


def cache(p):
    return A.PagedCache(p, on(0, 5, HKV, PAGE, D), on(0, 5, HKV, PAGE, D))


def norm_args(**other):
    x = dict(q=on(0, T, H, D), k=on(0, T, HKV, D), positions=on(0, T, dtype=I32), rope=on(0, 9, D, dtype=F32),
             g_q=on(0, D, dtype=F32), g_k=on(0, D, dtype=F32), q_out=on(0, T, H, D), k_out=on(0, T, HKV, D))
    return {**x, **other}


def append_args(**other):
    x = dict(batch=batch(), k=on(0, T, HKV, D), v=on(0, T, HKV, D), rope=on(0, 9, D, dtype=F32), g_k=on(0, D, dtype=F32),
             q=on(0, T, H, D), g_q=on(0, D, dtype=F32), q_out=on(0, T, H, D))
    return {**x, **other}


def attend_args(**other):
    x = dict(batch=batch(), q=on(0, T, H, D), out=on(0, T, H, D), lse=on(0, T, H, dtype=F32),
             workspace=on(0, 1 << 16, dtype=torch.uint8))
    return {**x, **other}


def verify_args(**other):
    x = dict(target=on(0, B, 3, 10, dtype=F32), drafts=on(0, B, 2, dtype=I32), u=on(0, B, 3, dtype=F32),
             draft_probs=on(0, B, 2, 10, dtype=F32), n_drafts=on(0, B, dtype=I32), tokens=on(0, B, 3, dtype=I32),
             accepted=on(0, B, dtype=I32))
    return {**x, **other}


def calls():
    """(name in the library, the call, its tensors)."""
    p = plan()
    c = cache(p)
    return {"engram_qk_norm_rope": (p.qk_norm_rope, norm_args), "engram_kv_append": (c.append, append_args),
            "engram_paged_attention": (c.attend, attend_args), "engram_verify_drafts": (A.verify_drafts, verify_args)}


NAMES = [(n, k) for n, args in (("engram_qk_norm_rope", norm_args), ("engram_kv_append", append_args),
                                ("engram_paged_attention", attend_args), ("engram_verify_drafts", verify_args))
         for k in args()]


def moved(x):
    """The same on GPU 1."""
    return batch(1) if isinstance(x, A.SequenceBatch) else on(1, *x.shape, dtype=x.dtype)


@pytest.mark.parametrize("name,arg", NAMES)
def test_tensors_of_another_device_are_refused(lib, name, arg):
    call, args = calls()[name]
    call(**args())
    assert [n for n, _ in lib.calls].count(name) == 1
    with pytest.raises(ValueError, match="cuda:1"):
        call(**args(**{arg: moved(args()[arg])}))
    assert [n for n, _ in lib.calls].count(name) == 1


def test_caches_and_batches_are_on_one_device(lib):
    p = plan()
    good = on(0, 5, HKV, PAGE, D)
    for k, v in ((good, moved(good)), (moved(good), good)):
        with pytest.raises(ValueError, match="cuda:1"):
            A.PagedCache(p, k, v)
    start, length, table = on(0, B + 1, dtype=I32), on(0, B, dtype=I32), on(0, B, 3, dtype=I32)
    for x in ((moved(start), length, table), (start, moved(length), table), (start, length, moved(table))):
        with pytest.raises(ValueError, match="cuda:1"):
            A.SequenceBatch(*x)


def test_a_check_of_drafts_runs_on_the_current_device(lib, monkeypatch):
    everything = {k: moved(v) for k, v in verify_args().items()}
    with pytest.raises(ValueError, match="cuda:1"):
        A.verify_drafts(**everything)
    monkeypatch.setattr(A, "_current_device", lambda: 1)
    A.verify_drafts(**everything)
    assert [n for n, _ in lib.calls] == ["engram_verify_drafts"]


def test_the_plans_own_workspace_is_on_its_device(lib, monkeypatch):
    """Also where another device is current, whose default stream has the same handle."""
    p = plan()
    p.device = 1
    made = []
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: made.append(device) or torch.zeros(1 << 16, dtype=torch.uint8))
    p.new_workspace()
    p._workspace(0)
    assert made == [torch.device("cuda", 1)] * 2


@pytest.mark.parametrize("name,arg", [(n, k) for n, k in NAMES if k in ("q", "k", "v", "rope", "g_q", "g_k", "target",
                                                                       "draft_probs", "u")])
def test_inputs_that_require_a_gradient_are_refused(lib, name, arg):
    call, args = calls()[name]
    x = args()
    x[arg].requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        call(**x)
    assert name not in [n for n, _ in lib.calls]
    with torch.no_grad():
        call(**x)
    with torch.inference_mode():
        call(**x)
    assert [n for n, _ in lib.calls].count(name) == 2


@pytest.mark.parametrize("window,passed", [(0, 0), (7, 7), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1),
                                           (2 ** 32 + 5, 2 ** 31 - 1), (2 ** 63 - 1, 2 ** 31 - 1)])
def test_windows_of_any_size_reach_the_library(lib, window, passed):
    """One longer than any sequence is not cut to its low 32 bits."""
    call, args = calls()["engram_paged_attention"]
    call(**args(), window=window)
    name, at = lib.calls[-1]
    assert name == "engram_paged_attention" and at[4] == passed


@pytest.mark.parametrize("scale", [0.0, -1.0, float("nan"), 1e-50])
def test_scales_that_are_not_positive_floats_are_refused(lib, scale):
    """1e-50 is 0 as a float32, which would stand for the default scale."""
    with pytest.raises(ValueError, match="scale"):
        A.AttentionPlan(heads=H, heads_kv=HKV, head_dim=D, scale=scale)
    assert lib.calls == []


@pytest.mark.parametrize("name,args", [("append", append_args), ("attend", attend_args)])
def test_a_cache_of_a_closed_plan_is_refused(lib, name, args):
    """The cache's handle points at the plan's."""
    p = plan()
    c = cache(p)
    getattr(c, name)(**args())
    p.close()
    n = len(lib.calls)
    with pytest.raises(ValueError, match="closed"):
        getattr(c, name)(**args())
    assert len(lib.calls) == n
