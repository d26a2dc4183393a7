"""Host threads that raise a kernel's shared-memory limit at the same time (CPU: the two driver calls are stand-ins)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <mutex>
#include <thread>

#include "smem_limit.cuh"

// The driver: a limit per device. A call that asks for 200 KB is held up until another call has been answered, or 200 ms.
static int limit[2] = {48, 48};
static thread_local int device = 0;
static std::mutex mu;
static std::condition_variable cv;
static bool large_in = false, small_done = false;

extern "C" cudaError_t CUDARTAPI cudaGetDevice(int* d) {
  *d = device;
  return cudaSuccess;
}
extern "C" cudaError_t CUDARTAPI cudaFuncSetAttribute(const void*, enum cudaFuncAttribute, int value) {
  std::unique_lock<std::mutex> lk(mu);
  limit[device] = value;
  if (value == 200) {
    large_in = true;
    cv.notify_all();
    cv.wait_for(lk, std::chrono::milliseconds(200), [] { return small_done; });
  } else {
    small_done = true;
    cv.notify_all();
  }
  return cudaSuccess;
}

static void kernel() {}

int main() {
  std::thread a([] { moe::allow_smem<kernel>(200); });
  std::thread b([] {
    {
      std::unique_lock<std::mutex> lk(mu);
      cv.wait(lk, [] { return large_in; });
    }
    moe::allow_smem<kernel>(100);
  });
  a.join();
  b.join();
  // A launch that needs 200 comes after both.
  if (moe::allow_smem<kernel>(200) != MOE_OK) return 2;
  std::printf("%d", limit[0]);
  device = 1;
  moe::allow_smem<kernel>(150);
  moe::allow_smem<kernel>(120);
  std::printf(" %d", limit[1]);
  return 0;
}
"""


def test_a_smaller_request_beside_a_larger_one(tmp_path):
    cxx, cuda = shutil.which("g++") or shutil.which("c++"), "/usr/local/cuda/include"
    if cxx is None or not os.path.exists(os.path.join(cuda, "cuda_runtime_api.h")):
        pytest.skip("no C++ compiler or CUDA headers")
    src, exe = tmp_path / "limit.cpp", tmp_path / "limit"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-pthread", "-x", "c++", "-I", cuda, "-I", os.path.join(ROOT, "serving_router_softmax_gb300", "csrc"),
                    "-o", str(exe), str(src)], check=True)
    assert subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60).stdout == "200 150"
