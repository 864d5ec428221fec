"""What the launch helpers of the operators around the projections report, against a fake of the CUDA runtime that
keeps a failed call's error, as the runtime does, until it is asked for the last one."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <stdio.h>
#include <string.h>

#include "block.h"

// the fake: `next` is what the next call returns, `last` what a failed one left behind
static cudaError_t next = cudaSuccess, last = cudaSuccess;
static int attributes = -1, limit = -1, value = 0;
static cudaError_t call() {
  const cudaError_t e = next;
  if (e != cudaSuccess) last = e;
  next = cudaSuccess;
  return e;
}
extern "C" {
cudaError_t cudaGetDevice(int *d) { *d = 0; return call(); }
cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int v) { limit = v; return call(); }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *, void **args) {
  attributes = static_cast<int>(c->numAttrs);
  value = *static_cast<int *>(args[0]);
  return call();
}
cudaError_t cudaGetLastError(void) { const cudaError_t e = last; last = cudaSuccess; return e; }
}

static void kern(int) {}
static int bad = 0;
static void check(bool ok, const char *what) {
  if (!ok) printf("%s\n", what), bad = 1;
}

int main() {
  using namespace svdq;
  const dim3 grid(3);
  auto dependent = [&] { return launch_dependent(kern, grid, 64, 0, nullptr, 17); };
  auto in_order = [&] { return launch(kern, grid, 64, 0, nullptr, 18); };
  auto allow = [&] { return allow_smem<65536>(kern); };
  check(dependent() == cudaSuccess && attributes == 1 && value == 17, "dependent launch");
  check(in_order() == cudaSuccess && attributes == 0 && value == 18, "launch in order");
  // a failure is the call's own, and leaves nothing for the next one to find
  next = cudaErrorInvalidValue;
  check(dependent() == cudaErrorInvalidValue && last == cudaSuccess, "failed dependent launch");
  next = cudaErrorInvalidConfiguration;
  check(in_order() == cudaErrorInvalidConfiguration && last == cudaSuccess, "failed launch in order");
  next = cudaErrorNoDevice;  // (cudaGetDevice)
  check(allow() == cudaErrorNoDevice && last == cudaSuccess, "no device");
  // an error that something else left behind is not these calls'
  last = cudaErrorMemoryAllocation;
  check(dependent() == cudaSuccess && in_order() == cudaSuccess, "another call's error");
  last = cudaSuccess;
  // the limit is set once, to the kernel's own
  check(allow() == cudaSuccess && limit == 65536, "limit");
  limit = -1;
  check(allow() == cudaSuccess && limit == -1, "limit remembered");
  check(allow_smem<40 * 1024>(kern) == cudaSuccess && limit == -1, "within the default");
  check(reported(cudaSuccess) == cudaSuccess, "success");
  printf(bad ? "failed\n" : "passed\n");
  return bad;
}
"""


def _cuda_include():
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")


def test_statuses_belong_to_their_calls(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None or not os.path.exists(os.path.join(_cuda_include(), "cuda_runtime.h")):
        pytest.skip("no host compiler or CUDA headers")
    src, exe = tmp_path / "launch.cpp", tmp_path / "launch"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++20", f"-isystem{_cuda_include()}", f"-I{ROOT}/include",
                    f"-I{ROOT}/bit_rank_compensated_b200/csrc", str(src), "-o", str(exe)], check=True, timeout=300)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "passed\n", r.stdout
