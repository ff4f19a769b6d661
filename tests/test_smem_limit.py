"""Two host threads whose first calls of a kernel ask for different amounts of
dynamic shared memory (the amount grows with the number of sequences): the one
that asks for more must find its limit set when it launches.  The library's
class runs on the CPU, on stand-ins for the two CUDA calls that it makes."""

import subprocess

from exact_attention_fattn_gb300 import build

PROGRAM = r"""
#include "fattn_smem_limit.h"

#include <chrono>
#include <cstdio>
#include <thread>

static std::atomic<int> limit{0}, in_small{0}, large_done{0}, small_set{0}, looked{0};
static void wait_for(const std::atomic<int>& flag) {   // or a third of a second
  for (int i = 0; i < 300 && !flag; ++i) std::this_thread::sleep_for(std::chrono::milliseconds(1));
}

extern "C" cudaError_t cudaGetDevice(int* dev) {
  *dev = 0;
  return cudaSuccess;
}

// The small request takes effect only when the large one has returned, and
// returns only when the large one's thread has looked at the limit; both only
// where that thread does not wait for this one.
extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int bytes) {
  if (bytes == 1000) {
    in_small = 1;
    wait_for(large_done);
  }
  limit = bytes;
  if (bytes == 1000) {
    small_set = 1;
    wait_for(looked);
  }
  return cudaSuccess;
}

int main() {
  static fattn::SmemLimit kernel;
  static int seen = 0;
  std::thread small([] { kernel.raise(nullptr, 1000); });
  std::thread large([] {
    wait_for(in_small);
    kernel.raise(nullptr, 2000);
    large_done = 1;
    wait_for(small_set);
    seen = limit;           // what a launch would find
    looked = 1;
  });
  small.join();
  large.join();
  kernel.raise(nullptr, 500);
  std::printf("%d %d\n", seen, limit.load());
  return seen >= 2000 && limit >= 2000 ? 0 : 1;
}
"""


def test_a_smaller_request_does_not_lower_another_threads_limit(tmp_path):
    src, exe = tmp_path / "limit.cpp", tmp_path / "limit"
    src.write_text(PROGRAM)
    subprocess.run([build._nvcc(), "-std=c++17", "-cudart", "none", "-I", build.CSRC, str(src), "-o", str(exe),
                    "-Xcompiler", "-pthread"], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
