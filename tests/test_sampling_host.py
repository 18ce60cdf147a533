"""Arithmetic of sampling that the settings' whole range reaches, compiled from the library's own header for the
host with nvcc and gcc's checks of undefined behaviour."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "hashed_gram_embedding_engram_gb300", "csrc")

PROGRAM = r'''
#include <climits>
#include <cstdio>
#include "sample_parts.cuh"
int main() {
  int bad = 0;
  const int ks[] = {INT_MIN, -7, 0, 1, 2, 7, 8, 9, 50, 1000, 32003, 129280, 1 << 24, 1 << 30, INT_MAX - 7, INT_MAX - 1, INT_MAX};
  const int vs[] = {1, 2, 31, 900, 32003, 129280, 1 << 24};
  for (int k : ks)
    for (int V : vs)
      for (int blocks = 1; blocks <= 8; ++blocks) {
        const long long kept = k < 0 ? 0 : (k < V ? k : V);
        const int got = engram::sample::top_k_share(k, V, blocks);
        if (got != (kept + blocks - 1) / blocks && bad++ < 10)
          std::printf("FAIL top_k %d V %d blocks %d got %d\n", k, V, blocks, got);
      }
  std::printf("bad %d\n", bad);
  return bad != 0;
}
'''


@pytest.mark.timeout(600)
def test_a_blocks_share_of_any_top_k(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    src, exe = tmp_path / "share.cu", tmp_path / "share"
    src.write_text(PROGRAM)
    subprocess.run([nvcc, "-std=c++17", "-O1", "-I", CSRC, "-gencode", "arch=compute_103a,code=sm_103a",
                    "-Xcompiler", "-fsanitize=undefined,-fno-sanitize-recover", str(src), "-lubsan", "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and "bad 0" in r.stdout, r.stdout + r.stderr
