"""How attention cuts its line of steps among the blocks (attn_sched.cuh, Cut), compiled from the
library's own header for the host with nvcc and checked against whole-number division: in 32 bits,
at their end, and in 64, which only calls of 2^31 steps and more take."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "hashed_gram_embedding_engram_gb300", "csrc")

PROGRAM = r'''
#include <cstdio>
#include "attn_sched.cuh"
using namespace engram::at;
static long long checked = 0;
static int bad = 0;
static int64_t exact(int64_t c, int64_t U, int C) { return static_cast<int64_t>(static_cast<__int128>(c) * U / C); }
static void find(const Cut& g, int64_t u) {
  if (u < 0 || u >= g.U) return;
  const int c = cut_find(g, u);
  const bool ok = c >= 0 && c < g.C && exact(c, g.U, g.C) <= u && u < exact(c + 1, g.U, g.C);
  ++checked;
  if (!ok && bad++ < 10) std::printf("FAIL U=%lld C=%d u=%lld got %d\n", (long long)g.U, g.C, (long long)u, c);
}
static void cut(int64_t U, int C, bool all) {
  const Cut g = make_cut(U, C);
  for (int c = 0; c <= C; ++c) {
    const int64_t at = cut_begin(g, c);
    ++checked;
    if (at != exact(c, U, C) && bad++ < 10)
      std::printf("FAIL U=%lld C=%d begin(%d) = %lld\n", (long long)U, C, c, (long long)at);
    for (int64_t d = -2; d <= 2; ++d) find(g, at + d);
    find(g, at + U / C / 2);
  }
  for (int64_t u = 0; all && u < U; ++u) find(g, u);
}
int main() {
  const int blocks[] = {1, 2, 3, 7, 100, 151, 152, 304, 455, 608};
  for (int C : blocks) {
    for (int64_t U = C; U < C + 700; ++U) cut(U, C, true);
    for (int s = 10; s < 50; ++s)
      for (int64_t d = -3; d <= 3; ++d)
        if ((int64_t(1) << s) + d >= C) cut((int64_t(1) << s) + d, C, false);
    for (int64_t U = C; U < (int64_t(1) << 46); U = U * 3 + 1) cut(U, C, false);
  }
  std::printf("checked %lld bad %d\n", checked, bad);
  return bad != 0;
}
'''


@pytest.mark.timeout(600)
def test_ranges_tile_the_line_and_every_place_is_found(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    src, exe = tmp_path / "cut_check.cu", tmp_path / "cut_check"
    src.write_text(PROGRAM)
    subprocess.run([nvcc, "-std=c++17", "-O2", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
                    "-gencode", "arch=compute_103a,code=sm_103a", str(src), "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and "bad 0" in r.stdout, r.stdout + r.stderr
