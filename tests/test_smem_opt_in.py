"""The shared-memory opt-in of the kernels, called by several host threads at once, against a stand-in for the
CUDA runtime: no GPU."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "binarized_transformer_b200", "csrc")

PROGRAM = r"""
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <mutex>
#include <thread>

#include "smem_opt_in.h"

// The stand-in: one attribute; the call that sets HOLD returns late, when another size has been set since or
// a while has passed.
constexpr int HOLD = 40960;
std::mutex m;
std::condition_variable cv;
int attribute = 0, calls = 0;
bool failing = false;

extern "C" cudaError_t cudaGetDevice(int *device) {
  *device = 0;
  return cudaSuccess;
}
extern "C" cudaError_t cudaFuncSetAttribute(const void *, enum cudaFuncAttribute attr, int value) {
  if (attr != cudaFuncAttributeMaxDynamicSharedMemorySize) return cudaSuccess;
  std::unique_lock<std::mutex> lock(m);
  if (failing) return cudaErrorInvalidValue;
  attribute = value;
  ++calls;
  cv.notify_all();
  if (value == HOLD) cv.wait_for(lock, std::chrono::milliseconds(500), [] { return attribute != HOLD; });
  return cudaSuccess;
}
void kernel() {}

int main() {
  static bwta::SmemOptIn opt;
  failing = true;
  if (opt(kernel, 1000) != cudaErrorInvalidValue) return std::puts("an error was lost"), 1;
  failing = false;
  std::thread large([] { opt(kernel, HOLD); });
  {
    std::unique_lock<std::mutex> lock(m);
    cv.wait(lock, [] { return attribute == HOLD; });
  }
  std::thread small([] { opt(kernel, 20480); });  // while the larger call is under way
  large.join();
  small.join();
  if (opt(kernel, 32768) != cudaSuccess || attribute < 32768)
    return std::printf("launched with %d bytes on an attribute of %d\n", 32768, attribute), 1;
  const int before = calls;
  if (opt(kernel, HOLD) != cudaSuccess || calls != before) return std::puts("set again"), 1;
  if (opt(kernel, 2 * HOLD) != cudaSuccess || attribute != 2 * HOLD) return std::puts("not raised"), 1;
  return std::puts("ok"), 0;
}
"""


def test_a_smaller_size_never_replaces_a_larger_one(tmp_path):
    nvcc = shutil.which(os.environ.get("NVCC", "nvcc"))
    if nvcc is None:
        pytest.skip("no CUDA toolkit")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    src, exe = tmp_path / "opt_in.cpp", tmp_path / "opt_in"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", CSRC, "-I", include, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
