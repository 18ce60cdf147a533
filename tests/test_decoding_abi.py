"""The C ABI of trees, pages and sampling without a GPU: the host-side checks refuse before any CUDA
call; the oracle's own pins; plans on two devices."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

from oracle import decoding_oracle as O
from test_attention_abi import lib  # noqa: F401
from test_attention_devices import PROGRAM, ROOT

SOURCES = ["tree.cu", "pages.cu", "sample.cu", "sample_parts.cuh", "serving.cu", "attn_host.h"]


def test_null_handles_and_bad_sizes_are_refused(lib):  # noqa: F811
    from hashed_gram_embedding_engram_gb300 import _lib
    bad, n = _lib.ERR_INVALID_ARG, ctypes.c_size_t()
    assert lib.engram_tree_build(None, None, None, None, None) == bad
    assert lib.engram_tree_attention(None, None, None, None, None, None, None, 0, None) == bad
    assert lib.engram_tree_accept(None, None, None, None, None, 1, None, None, None, None, None) == bad
    assert lib.engram_kv_compact(None, None, None, 1, None, None) == bad
    assert lib.engram_kv_copy_pages(None, None, 1, None) == bad
    assert lib.engram_pool_free(None, None, None, None, 1, None) == bad
    assert lib.engram_pool_fork(None, None, None, None, None, 1, None) == bad
    assert lib.engram_pool_reserve(None, None, None, None, None, None, None, 0, None) == bad
    assert lib.engram_pool_workspace_bytes(None, ctypes.byref(n)) == bad
    s = lambda R, V, stride, t=_lib.F32, p=None: lib.engram_sample_tokens(p, t, stride, None, None, R, V, None, None)  # noqa: E731
    assert s(1, 10, 10, _lib.I8_ROWSCALE_F16) == _lib.ERR_UNSUPPORTED
    assert s(-1, 10, 10) == bad and s(2 ** 24, 10, 10) == bad and s(1, 0, 10) == bad and s(1, 2 ** 24 + 1, 2 ** 25) == bad
    assert s(1, 10, 9) == bad and s(2, 10, 2 ** 62) == bad and s(1, 10, 10) == bad
    assert s(0, 10, 10) == _lib.OK


@pytest.mark.parametrize("source", SOURCES)
def test_no_read_only_loads_under_programmatic_launch(source):
    """As for the attention kernels: what an earlier kernel may have written is not read by read-only loads."""
    from hashed_gram_embedding_engram_gb300 import build
    with open(os.path.join(build.CSRC, source)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert re.findall(r"__ldg|ld\.global\.nc|__restrict__", code) == []


PART = r'''
// Every new call of a plan belongs to the plan's device, and refuses what it cannot take before it launches.
static void decoding() {
  for (engram_dtype_t t : {ENGRAM_F32, ENGRAM_BF16}) {
    Layer x(t, 128, 0);
    engram_sequences_t s = {kInts, kInts, kInts, 1, 4, 4, 4};
    engram_tree_t tree = {(uint32_t*)kMem, (int32_t*)kMem, 2, 0};
    engram_pool_t pool = {(int32_t*)kMem, (int32_t*)kMem, 3, 4, 100};
    engram_sampling_t set = {nullptr, nullptr, nullptr, nullptr, 1.f, 0, 1.f, 0.f};
    int32_t* const out = (int32_t*)kMem;
    size_t bytes = 0;
    expect(engram_pool_workspace_bytes(&pool, &bytes) == ENGRAM_OK && bytes > 0, "pool workspace", 0, 0);
    auto calls = [&](engram_status_t want, const char* what) {
      const int before = g_launches;
      expect(engram_tree_build(x.plan, &s, kInts, &tree, nullptr) == want, what, 1, 0);
      expect(engram_tree_attention(x.cache, &s, &tree, &kView, kMem, nullptr, kMem, x.bytes, nullptr) == want, what, 2, 0);
      expect(engram_tree_accept(x.plan, &s, kInts, kInts, kInts, 8, out, out, out, out, nullptr) == want, what, 3, 0);
      expect(engram_kv_compact(x.cache, &s, kInts, 8, kInts, nullptr) == want, what, 4, 0);
      expect(engram_kv_compact(x.cache, &s, kInts, 800, kInts, nullptr) == want, what, 5, 0);
      expect(engram_kv_copy_pages(x.cache, kInts, 3, nullptr) == want, what, 6, 0);
      expect(engram_pool_free(x.plan, &pool, kInts, kInts, 2, nullptr) == want, what, 7, 0);
      expect(engram_pool_fork(x.plan, &pool, kInts, kInts, kInts, 2, nullptr) == want, what, 8, 0);
      expect(engram_pool_reserve(x.plan, &pool, kInts, kInts, out, out, kMem, bytes, nullptr) == want, what, 9, 0);
      if (want != ENGRAM_OK) expect(g_launches == before, "launches of refused calls", before, g_launches);
    };
    calls(ENGRAM_OK, "on the plan's device");
    g_device = 1;
    calls(ENGRAM_ERR_INVALID_ARG, "on another device");
    g_device = 0;
    const int before = g_launches;
    auto bad_tree = [&](engram_tree_t b) { return engram_tree_build(x.plan, &s, kInts, &b, nullptr) == ENGRAM_ERR_INVALID_ARG; };
    expect(bad_tree({nullptr, out, 2, 0}) && bad_tree({(uint32_t*)kMem, nullptr, 2, 0}) && bad_tree({(uint32_t*)kMem, out, 0, 0}) &&
           bad_tree({(uint32_t*)kMem, out, 9, 0}) && bad_tree({(uint32_t*)kMem, out, 2, -1}), "bad trees", 0, 0);
    expect(engram_tree_attention(x.cache, &s, &tree, &kView, kMem, nullptr, kMem, x.bytes - 1, nullptr) == ENGRAM_ERR_WORKSPACE,
           "small workspace", 0, 0);
    for (int width : {0, -1, 257})
      expect(engram_tree_accept(x.plan, &s, kInts, kInts, kInts, width, out, out, out, out, nullptr) == ENGRAM_ERR_INVALID_ARG,
             "width", width, 0);
    expect(engram_kv_compact(x.cache, &s, kInts, 0, kInts, nullptr) == ENGRAM_ERR_INVALID_ARG, "no columns", 0, 0);
    expect(engram_kv_copy_pages(x.cache, kInts, -1, nullptr) == ENGRAM_ERR_INVALID_ARG, "pairs", 0, 0);
    expect(engram_kv_copy_pages(x.cache, kInts, 1ll << 40, nullptr) == ENGRAM_ERR_UNSUPPORTED, "too many pairs", 0, 0);
    expect(engram_pool_free(x.plan, &pool, kInts, kInts, 65537, nullptr) == ENGRAM_ERR_UNSUPPORTED, "too many rows", 0, 0);
    for (engram_pool_t p : {engram_pool_t{nullptr, out, 3, 4, 100}, {out, nullptr, 3, 4, 100}, {out, out, -1, 4, 100},
                            {out, out, 3, 0, 100}, {out, out, 3, 1 << 25, 100}, {out, out, 3, 4, 0}, {out, out, 3, 4, 1ll << 31}})
      expect(engram_pool_free(x.plan, &p, kInts, kInts, 1, nullptr) == ENGRAM_ERR_INVALID_ARG &&
             engram_pool_reserve(x.plan, &p, kInts, kInts, out, out, kMem, bytes, nullptr) == ENGRAM_ERR_INVALID_ARG, "bad pools", 0, 0);
    expect(engram_pool_reserve(x.plan, &pool, kInts, kInts, out, out, kMem, bytes - 1, nullptr) == ENGRAM_ERR_WORKSPACE, "workspace", 0, 0);
    expect(g_launches == before, "launches of refused calls", before, g_launches);
    // sampling, around the sizes at which rows get other numbers of blocks, aligned and not
    for (long long V : {1ll, 100ll, 1000ll, 32003ll, 129280ll, 600001ll, 1ll << 24})
      for (long long R : {1ll, 20ll, 300ll, 5000ll})
        expect(engram_sample_tokens((char*)kMem + 4, t, V, (const float*)kMem, &set, R, V, out, nullptr) == ENGRAM_OK, "sampling",
               (int)V, (int)R);
    expect(engram_sample_tokens((char*)kMem + 1, t, 10, (const float*)kMem, &set, 1, 10, out, nullptr) == ENGRAM_ERR_INVALID_ARG,
           "unaligned logits", 0, 0);
    const int none = g_launches;
    s.tokens = 0;
    expect(engram_tree_build(x.plan, &s, nullptr, nullptr, nullptr) == ENGRAM_OK && g_launches == none, "no tokens", 0, 0);
    s.B = 0;
    expect(engram_tree_accept(x.plan, &s, nullptr, nullptr, nullptr, 8, nullptr, nullptr, nullptr, nullptr, nullptr) == ENGRAM_OK &&
           engram_kv_compact(x.cache, &s, nullptr, 8, nullptr, nullptr) == ENGRAM_OK && g_launches == none, "no sequences", 0, 0);
  }
}
'''


def test_calls_refuse_other_devices_and_bad_arguments(tmp_path):
    """With the stand-in for the CUDA runtime of test_attention_devices.py, which refuses a launch whose shared
    memory was not allowed on its device."""
    from hashed_gram_embedding_engram_gb300 import build
    build.build()
    head, main = PROGRAM.split("int main(")
    program = head + PART + "int main(" + main.replace('if (!strcmp(argv[1], "other"))', 'if (!strcmp(argv[1], "decoding")) decoding();\n  if (!strcmp(argv[1], "other"))')
    objects = [os.path.join(build.BUILD, f"{n}.o") for n in
               ("attention", "attn_rows", "attn_tiles", "attn_simt", "rope", "verify", "serving", "tree", "pages", "sample")]
    src, exe = tmp_path / "decoding.cpp", tmp_path / "decoding"
    src.write_text(program)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc())))
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", build.CSRC, "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(cuda, "include"), str(src), *objects, "-ldl", "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    for scenario in ("decoding", "other"):
        r = subprocess.run([str(exe), scenario], capture_output=True, text=True, timeout=60)
        assert r.returncode == 0 and "bad 0" in r.stdout, r.stdout + r.stderr


# ---------------------------------------------------------------- the oracle's own pins
def test_oracle_layout_by_hand():
    sees, at = O.layout([-1, 0, 0, 1, -1, 3], [0, 6], [20])
    assert at.tolist() == [14, 15, 15, 16, 14, 17]
    assert [np.flatnonzero(r).tolist() for r in sees[0]] == [[0], [0, 1], [0, 2], [0, 1, 3], [4], [0, 1, 3, 5]]
    sees, _ = O.layout([-1, 0, 0, 1, -1, 3], [0, 6], [20], window=2)
    assert np.flatnonzero(sees[0][5]).tolist() == [3, 5]
    sees, at = O.layout([-1, 0, 5, 2, 1], [0, 5], [9])
    assert not sees[0][2:4].any() and at.tolist() == [4, 5, 0, 0, 6]
    assert not O.layout([-1, 0], [0, 2], [1])[0][0].any()


def test_oracle_path_by_hand():
    path, count, out, length = O.accept([-1, 0, 0, 1, 2, 2], [9, 5, 6, 7, 8, 8], [6, 1, 8, 2, 3, 4], [0, 6], [30], 4)
    assert path.tolist() == [[0, 2, 4, -1]] and out.tolist() == [[6, 8, 3, -1]] and count.tolist() == [3] and length.tolist() == [27]


def test_oracle_weights_and_filters_by_hand():
    assert O.weights(np.float32([3, 3, -np.inf, np.nan]), 1.0) == [2 ** 38, 2 ** 38, 0, 0]
    w = O.weights(np.float32([0, -math_ln2(1), -math_ln2(3)]), 1.0)
    assert w[0] == 2 ** 38 and abs(w[1] / 2 ** 37 - 1) < 1e-6 and abs(w[2] / 2 ** 35 - 1) < 1e-6
    l = np.float32([1, 4, 4, 2, 4])
    assert sorted(O.kept(l, top_k=2)) == [1, 2] and sorted(O.kept(l, temperature=0)) == [1]
    assert sorted(O.kept(l, top_p=0.5)) == [1, 2] and sorted(O.kept(l, top_p=0.0)) == [1]
    assert sorted(O.kept(l, min_p=0.5)) == [1, 2, 4]
    assert [O.sample(l, u, top_k=3) for u in (0.0, 0.34, 0.99)] == [1, 2, 4]


def math_ln2(n):
    return n * float(np.log(2.0))


def test_oracle_pool_by_hand():
    p = O.Pool([[0, 1, -1], [-1, -1, -1]], [1, 1, 0, 0], 16)
    p.fork([0], [1], [20])
    assert p.table[1] == [0, 1, -1] and p.ref == [2, 2, 0, 0]
    assert p.reserve([20, 20], [21, 20]) == ([[1, 2], [-1, -1]], 0) and p.ref == [2, 1, 1, 0]
    p.free([1], [16])
    assert p.table[1] == [0, -1, -1] and p.ref == [2, 0, 1, 0]
    assert p.reserve([21, 0], [48, 48])[1] == 2
