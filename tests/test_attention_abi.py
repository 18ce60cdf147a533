"""engram_attention.h without a GPU: the host-side checks refuse before any CUDA call, and the
oracle's own pins."""
import ctypes
import os
import re

import numpy as np
import pytest

from oracle import attention_oracle as O


@pytest.fixture(scope="module")
def lib():
    from hashed_gram_embedding_engram_gb300 import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib._lib()


@pytest.mark.parametrize("bad", [dict(heads=0), dict(heads=5), dict(heads_kv=0), dict(heads=1032, heads_kv=8),
                                 dict(heads=512, heads_kv=2), dict(head_dim=0), dict(head_dim=20), dict(head_dim=264),
                                 dict(page=0), dict(page=4), dict(page=48), dict(page=2048), dict(rotary_dim=-16),
                                 dict(rotary_dim=8), dict(rotary_dim=144), dict(eps=0.0), dict(eps=float("nan")),
                                 dict(scale=-1.0), dict(scale=float("inf"))])
def test_plan_rejects_bad_shapes_before_cuda(lib, bad):
    from hashed_gram_embedding_engram_gb300 import _lib
    c = dict(heads=8, heads_kv=2, head_dim=128, page=16, dtype=_lib.BF16, rotary_dim=128, rope_adjacent=0, eps=1e-6,
             scale=0.0)
    c.update(bad)
    h = ctypes.c_void_p()
    cfg = _lib.AttnConfig(*[c[n] for n, _ in _lib.AttnConfig._fields_])
    assert lib.engram_attn_plan_create(ctypes.byref(cfg), ctypes.byref(h)) == _lib.ERR_INVALID_ARG
    assert not h.value


def test_plan_rejects_other_types_before_cuda(lib):
    from hashed_gram_embedding_engram_gb300 import _lib
    h = ctypes.c_void_p()
    cfg = _lib.AttnConfig(8, 2, 128, 16, _lib.I8_ROWSCALE_F16, 128, 0, 1e-6, 0.0)
    assert lib.engram_attn_plan_create(ctypes.byref(cfg), ctypes.byref(h)) == _lib.ERR_UNSUPPORTED


def test_null_handles_and_bad_sizes_are_refused(lib):
    from hashed_gram_embedding_engram_gb300 import _lib
    bad, h, n = _lib.ERR_INVALID_ARG, ctypes.c_void_p(), ctypes.c_size_t()
    assert lib.engram_attn_plan_create(None, ctypes.byref(h)) == bad
    assert lib.engram_attn_plan_destroy(None) == _lib.OK
    assert lib.engram_attn_get_error(None, None, None) == bad
    assert lib.engram_attn_workspace_bytes(None, ctypes.byref(n)) == bad
    assert lib.engram_kv_cache_create(None, None, None, 1, ctypes.byref(h)) == bad
    assert lib.engram_kv_cache_destroy(None) == _lib.OK
    assert lib.engram_qk_norm_rope(None, None, None, 1, None, None, 0, None, None, None, None, None) == bad
    assert lib.engram_kv_append(None, None, None, None, None, 0, None, None, None, None, None) == bad
    assert lib.engram_paged_attention(None, None, None, 1, 0, None, None, None, 0, None) == bad
    v = lambda B, S, V, d=_lib.F32: lib.engram_verify_drafts(None, None, d, None, None, None, B, S, V, None, None, None)  # noqa: E731
    assert v(1, 1, 10) == bad and v(-1, 1, 10) == bad and v(1, 0, 10) == bad and v(1, 65, 10) == bad
    assert v(1, 1, 0) == bad and v(1, 1, 2 ** 24 + 1) == bad and v(65536, 1, 10) == bad
    assert v(1, 1, 10, _lib.I8_ROWSCALE_F16) == _lib.ERR_UNSUPPORTED
    assert v(0, 1, 10) == _lib.OK


def test_oracle_rotation_keeps_norms_and_relative_angles():
    r = np.random.RandomState(0)
    D, L = 16, 40
    inv = 10000.0 ** (-np.arange(0, D, 2) / D)
    ang = np.arange(L)[:, None] * inv
    rope = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    q, k = r.randn(1, 1, D), r.randn(1, 1, D)
    for adjacent in (False, True):
        turn = lambda x, p: O.norm_rope(x, None, 1e-6, [p], rope, adjacent)[0, 0]  # noqa: E731
        assert np.isclose(np.linalg.norm(turn(q, 7)), np.linalg.norm(q))
        assert np.isclose(turn(q, 30) @ turn(k, 10), turn(q, 25) @ turn(k, 5))


def test_oracle_attention_of_equal_keys_is_the_mean_of_the_values():
    k, v = np.zeros((2, 1, 8, 8)), np.random.RandomState(1).randn(2, 1, 8, 8)
    q = np.random.RandomState(2).randn(2, 1, 8)
    out, lse, _ = O.attention(q, k, v, [0, 2], [11], np.array([[1, 0]]), 1.0)
    flat = np.concatenate([v[1, 0], v[0, 0]])
    assert np.allclose(out[0, 0], flat[:10].mean(0)) and np.allclose(out[1, 0], flat[:11].mean(0))
    assert np.allclose(lse[:, 0], np.log([10, 11]))
    out, lse, _ = O.attention(q, k, v, [0, 2], [11], np.array([[1, 0]]), 1.0, window=3)
    assert np.allclose(out[1, 0], flat[8:11].mean(0))


def test_oracle_verify_draws_the_target_distribution():
    """Over a grid of random numbers, the first token is distributed as the target."""
    p, q = np.array([0.5, 0.25, 0.25, 0.0]), np.array([0.25, 0.25, 0.25, 0.25])
    target = np.broadcast_to(p, (1, 2, 4)).astype(np.float64)
    count, m = np.zeros(4), 40
    for x in range(4):
        for i in range(m):
            for j in range(m):
                t, _ = O.verify(target, q[None, None], np.array([[x]]), None, np.array([[(i + .5) / m, (j + .5) / m]]))
                count[t[0, 0]] += q[x]
    assert np.allclose(count / (m * m), p, atol=1e-9)


@pytest.mark.parametrize("source", ["attn_rows.cu", "attn_tiles.cu", "attn_simt.cu", "attn_sched.cuh", "attn_tma.cuh",
                                    "rope.cu", "verify.cu"])
def test_no_read_only_loads_under_programmatic_launch(source):
    """These kernels start while the one before them may still write their inputs (the append the
    queries and pages, a projection all of them): a read-only load, or a const __restrict__ pointer
    of which the compiler may make one, is for memory that is not written meanwhile."""
    from hashed_gram_embedding_engram_gb300 import build
    with open(os.path.join(build.CSRC, source)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert re.findall(r"__ldg|ld\.global\.nc|__restrict__", code) == []
