"""Kernel settings made at first use, without a GPU: the helper compiled against a cudaGetDevice of
the test's own."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include "first_use.cuh"
#include <chrono>
#include <cstdio>
#include <thread>

static thread_local int device = 0;
extern "C" cudaError_t cudaGetDevice(int* d) {
  *d = device;
  return device < 0 ? cudaErrorNoDevice : cudaSuccess;
}

int main() {
  // threads that come while another one's setting takes its time: none goes on before it is made
  std::atomic<unsigned long long> flag{0};
  std::atomic<int> made{0}, early{0};
  auto slow = [&] {
    std::this_thread::sleep_for(std::chrono::milliseconds(200));
    ++made;
    return cudaSuccess;
  };
  auto use = [&] {
    if (pwp::on_first_use(flag, slow) != cudaSuccess || made == 0) ++early;
  };
  std::thread a(use);
  std::this_thread::sleep_for(std::chrono::milliseconds(50));
  std::thread b(use);
  a.join();
  b.join();
  if (early) return printf("a thread went on before the setting was made\n"), 1;
  const int once = made;
  use();
  if (made != once) return printf("set again\n"), 1;
  // another device has its own; one past the flag word sets every time
  device = 63;
  use(), use();
  if (made != once + 1) return printf("device 63 set %d times\n", made - once), 1;
  device = 64;
  use(), use();
  if (made != once + 3) return printf("device 64 set %d times\n", made - once - 1), 1;
  // a setting that failed is made again, and its error is the caller's
  std::atomic<unsigned long long> other{0};
  int tries = 0;
  device = 1;
  auto fails_once = [&] { return ++tries == 1 ? cudaErrorMemoryAllocation : cudaSuccess; };
  if (pwp::on_first_use(other, fails_once) != cudaErrorMemoryAllocation) return printf("error lost\n"), 1;
  if (pwp::on_first_use(other, fails_once) != cudaSuccess || tries != 2) return printf("not made again\n"), 1;
  pwp::on_first_use(other, fails_once);
  if (tries != 2) return printf("made three times\n"), 1;
  device = -1;
  if (pwp::on_first_use(other, fails_once) != cudaErrorNoDevice || tries != 2) return printf("no device\n"), 1;
  return 0;
}
"""


def test_nobody_launches_before_the_setting_is_made(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    if shutil.which("g++") is None or not os.path.exists(os.path.join(cuda, "include", "cuda_runtime_api.h")):
        pytest.skip("no C++ compiler or CUDA headers")
    src, exe = tmp_path / "first.cpp", tmp_path / "first"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-pthread", "-I", os.path.join(ROOT, "post_weight_pruning_b200", "csrc"), "-I",
                    os.path.join(cuda, "include"), str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
