"""The limit of dynamic shared memory is a setting of each device: raised on
every device that launches a kernel, and asked for again after a failure.  The
header that does it runs here over stand-ins for the two CUDA calls."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "neural_net_step_gb300", "csrc")

PROGRAM = r"""
#include "smem_limit.h"
#include <cstdio>
#include <thread>
#include <vector>
static thread_local int device = 0;
static int calls = 0, refuse = 0;
static std::map<std::pair<int, const void*>, int> limit;   // what each device has
cudaError_t cudaGetDevice(int* d) {
  if (device < 0) return cudaErrorNoDevice;
  *d = device;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v) {
  ++calls;
  if (refuse || a != cudaFuncAttributeMaxDynamicSharedMemorySize) return cudaErrorInvalidValue;
  limit[{device, f}] = v;
  return cudaSuccess;
}
#define CHECK(c) do { if (!(c)) { printf("line %d: %s\n", __LINE__, #c); return 1; } } while (0)
int main() {
  static char f, g;
  using mlpk::allow_smem;
  CHECK(allow_smem(&f, 48 * 1024) == cudaSuccess && calls == 0);          // within the limit there is
  CHECK(allow_smem(&f, 200000) == cudaSuccess && calls == 1 && (limit[{0, &f}] == 200000));
  CHECK(allow_smem(&f, 200000) == cudaSuccess && allow_smem(&f, 100000) == cudaSuccess && calls == 1);
  CHECK(allow_smem(&f, 220000) == cudaSuccess && calls == 2 && (limit[{0, &f}] == 220000));
  CHECK(allow_smem(&g, 100000) == cudaSuccess && calls == 3 && (limit[{0, &g}] == 100000));
  device = 1;                                                             // another device has limits of its own
  CHECK(allow_smem(&f, 200000) == cudaSuccess && calls == 4 && (limit[{1, &f}] == 200000));
  device = 2;
  refuse = 1;                                                             // a failure is returned, and not remembered
  CHECK(allow_smem(&f, 200000) == cudaErrorInvalidValue && allow_smem(&f, 200000) == cudaErrorInvalidValue && calls == 6);
  refuse = 0;
  CHECK(allow_smem(&f, 200000) == cudaSuccess && calls == 7 && (limit[{2, &f}] == 200000));
  device = -1;
  CHECK(allow_smem(&f, 200000) == cudaErrorNoDevice && calls == 7);
  std::vector<std::thread> t;                                             // several threads, a device each
  for (int d = 3; d < 11; ++d)
    t.emplace_back([d] {
      device = d;
      for (unsigned b = 60000; b < 61000; ++b) allow_smem(&f, b);
    });
  for (auto& x : t) x.join();
  for (int d = 3; d < 11; ++d) CHECK((limit[{d, &f}] == 60999));
  return 0;
}
"""


def test_limit_is_raised_on_every_device(tmp_path):
    nvcc = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    if not (shutil.which("g++") and os.path.exists(os.path.join(include, "cuda_runtime_api.h"))):
        pytest.skip("no C++ compiler or CUDA headers")
    src, exe = tmp_path / "limit.cpp", tmp_path / "limit"
    src.write_text(PROGRAM)
    r = subprocess.run(["g++", "-std=c++17", "-I", CSRC, "-I", include, str(src), "-o", str(exe), "-lpthread"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


def test_no_kernel_sets_its_limit_elsewhere():
    """Every launch goes through the header above: no other source sets the attribute."""
    for name in sorted(os.listdir(CSRC)):
        if name != "smem_limit.h":
            assert "MaxDynamicSharedMemorySize" not in open(os.path.join(CSRC, name)).read(), name
