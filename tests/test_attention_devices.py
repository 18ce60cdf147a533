"""Plans on several GPUs in one process, without a GPU: the library's own attention objects linked
with a stand-in for the CUDA runtime that has two devices, keeps what each was told about its
kernels, and refuses a launch as the runtime does."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r'''
#include <cuda_runtime_api.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <utility>

#include "attn_internal.h"

static int g_device = 0, g_launches = 0, g_syncs = 0, g_grid = 0;
static std::map<std::pair<const void*, int>, int> g_shared;   // bytes allowed to a kernel on a device

extern "C" {
cudaError_t CUDARTAPI cudaGetDevice(int* d) { *d = g_device; return cudaSuccess; }
cudaError_t CUDARTAPI cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int d) {
  *v = a == cudaDevAttrMultiProcessorCount ? (d == 0 ? 152 : 100) : a == cudaDevAttrComputeCapabilityMajor ? 10 : 3;
  return cudaSuccess;
}
cudaError_t CUDARTAPI cudaMalloc(void** p, size_t n) { *p = calloc(1, n); return cudaSuccess; }
cudaError_t CUDARTAPI cudaMemset(void* p, int v, size_t n) { memset(p, v, n); return cudaSuccess; }
cudaError_t CUDARTAPI cudaMemcpy(void* a, const void* b, size_t n, cudaMemcpyKind) { memcpy(a, b, n); return cudaSuccess; }
cudaError_t CUDARTAPI cudaFree(void* p) { free(p); return cudaSuccess; }
cudaError_t CUDARTAPI cudaStreamSynchronize(cudaStream_t) { ++g_syncs; return cudaSuccess; }
cudaError_t CUDARTAPI cudaGetLastError(void) { return cudaSuccess; }
cudaError_t CUDARTAPI cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v) {
  if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) g_shared[{f, g_device}] = v;
  return cudaSuccess;
}
cudaError_t CUDARTAPI cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void*, int, size_t, unsigned) {
  *n = g_device == 0 ? 2 : 1;
  return cudaSuccess;
}
cudaError_t CUDARTAPI cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  const auto at = g_shared.find({f, g_device});
  const size_t allowed = at == g_shared.end() ? 48 * 1024 : static_cast<size_t>(at->second);
  if (c->dynamicSmemBytes > allowed) return cudaErrorInvalidValue;
  ++g_launches;
  g_grid = static_cast<int>(c->gridDim.x);
  return cudaSuccess;
}
void** __cudaRegisterFatBinary(void*) { static void* h; return &h; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, void*, void*, void*, void*, int*) {}
cudaError_t __cudaPopCallConfiguration(void*, void*, size_t*, void*) { return cudaSuccess; }
cudaError_t __cudaGetKernel(void**, const void*) { return cudaSuccess; }
cudaError_t __cudaLaunchKernel(void*, dim3, dim3, void**, size_t, cudaStream_t) { return cudaSuccess; }
}
namespace engram {
bool make_tensor_map_2d(CUtensorMap*, const void*, bool, uint64_t, uint64_t, uint64_t, uint32_t, uint32_t, bool) {
  return true;
}
}

static int g_bad = 0;
static void expect(bool ok, const char* what, int a, int b) {
  if (!ok) std::printf("FAIL %s (%d, %d)\n", what, a, b), ++g_bad;
}

static void* const kMem = reinterpret_cast<void*>(0x100000);      // never touched: nothing runs
static const int32_t* const kInts = static_cast<const int32_t*>(kMem);
static const engram_heads_view_t kView = {kMem, 4096, 256};

struct Layer {
  engram_attn_plan_t* plan = nullptr;
  engram_kv_cache_t* cache = nullptr;
  size_t bytes = 0;
  Layer(engram_dtype_t t, int D, int device) {
    g_device = device;
    const engram_attn_config_t c = {8, 2, D, 64, t, 0, 0, 1e-6f, 0.f};
    expect(engram_attn_plan_create(&c, &plan) == ENGRAM_OK, "plan", D, device);
    engram_attn_workspace_bytes(plan, &bytes);
    expect(engram_kv_cache_create(plan, kMem, kMem, 16, &cache) == ENGRAM_OK, "cache", D, device);
  }
  engram_status_t norm() { return engram_qk_norm_rope(plan, &kView, nullptr, 4, nullptr, nullptr, 0, nullptr, nullptr, kMem, nullptr, nullptr); }
  engram_status_t append() {
    const engram_sequences_t s = {kInts, kInts, kInts, 1, 4, 4, 4};
    return engram_kv_append(cache, &s, &kView, &kView, nullptr, 0, nullptr, nullptr, nullptr, nullptr, nullptr);
  }
  engram_status_t attend(int n) {
    const engram_sequences_t s = {kInts, kInts, kInts, 1, 4, n, n};
    return engram_paged_attention(cache, &s, &kView, 1, 0, kMem, nullptr, kMem, bytes, nullptr);
  }
};

// Every call of a plan belongs to the plan's device: elsewhere it is refused and nothing starts.
static void other_device() {
  Layer x(ENGRAM_BF16, 128, 0);
  g_device = 1;
  const int before = g_launches;
  expect(x.norm() == ENGRAM_ERR_INVALID_ARG, "norm on another device", 0, 1);
  expect(x.append() == ENGRAM_ERR_INVALID_ARG, "append on another device", 0, 1);
  expect(x.attend(1) == ENGRAM_ERR_INVALID_ARG && x.attend(4) == ENGRAM_ERR_INVALID_ARG &&
         x.attend(100) == ENGRAM_ERR_INVALID_ARG, "attention on another device", 0, 1);
  expect(engram_attn_get_error(x.plan, nullptr, nullptr) == ENGRAM_ERR_INVALID_ARG && g_syncs == 0,
         "get_error on another device", 0, 1);
  expect(g_launches == before, "launches on another device", before, g_launches);
  g_device = 0;
  expect(x.norm() == ENGRAM_OK && x.append() == ENGRAM_OK && x.attend(1) == ENGRAM_OK &&
         engram_attn_get_error(x.plan, nullptr, nullptr) == ENGRAM_OK, "calls on the plan's device", 0, 0);
  expect(g_launches == before + 3, "launches on the plan's device", before, g_launches);
}

// Attention of every kernel and head size, on each device in turn.
static void each_device(int first) {
  for (int device : {first, 1 - first})
    for (int D : {8, 64, 96, 128, 256})
      for (engram_dtype_t t : {ENGRAM_F32, ENGRAM_BF16}) {
        Layer x(t, D, device);
        for (int n : {1, 5, 8, 100}) {
          expect(x.attend(n) == ENGRAM_OK, "attention", D, device);
          const int sms = device == 0 ? 152 : 100, per = device == 0 ? 2 : 1;
          if (t == ENGRAM_F32) expect(g_grid == sms * per, "blocks of a device", g_grid, device);
        }
      }
}

int main(int argc, char** argv) {
  if (!strcmp(argv[1], "other")) other_device();
  if (!strcmp(argv[1], "each01")) each_device(0);
  if (!strcmp(argv[1], "each10")) each_device(1);
  std::printf("bad %d\n", g_bad);
  return g_bad != 0;
}
'''


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    from hashed_gram_embedding_engram_gb300 import build
    build.build()
    objects = [os.path.join(build.BUILD, f"{n}.o") for n in
               ("attention", "attn_rows", "attn_tiles", "attn_simt", "rope", "verify")]
    where = tmp_path_factory.mktemp("devices")
    src, exe = where / "devices.cpp", where / "devices"
    src.write_text(PROGRAM)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc())))
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", build.CSRC, "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(cuda, "include"), str(src), *objects, "-ldl", "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    return str(exe)


def run(program, scenario):
    r = subprocess.run([program, scenario], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "bad 0" in r.stdout, r.stdout + r.stderr


def test_calls_with_another_device_current_are_refused(program):
    run(program, "other")


@pytest.mark.parametrize("order", ["each01", "each10"])
def test_attention_runs_on_every_device_that_has_a_plan(program, order):
    run(program, order)
