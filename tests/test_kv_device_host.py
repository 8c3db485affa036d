"""The attention's grid and workspace follow the current device, whichever came first: its header compiled against a CUDA
runtime of the test's own."""
import os
import subprocess

from quantized_weight_gb300 import build as qbuild

SOURCE = r"""
#include <cassert>
#include <cstdio>
#include <cstdlib>
#include <thread>
#include <vector>
#include "kv_attend.h"

static thread_local int device = 0;
static int sms[100] = {};
static int asked = 0;
static bool there = true;
extern "C" cudaError_t cudaGetDevice(int *d) { *d = device; return there ? cudaSuccess : cudaErrorNoDevice; }
extern "C" cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int d) {
  __atomic_fetch_add(&asked, 1, __ATOMIC_RELAXED);
  *v = sms[d];
  return cudaSuccess;
}
extern "C" cudaError_t cudaGetLastError() { return cudaSuccess; }

int main() {
  for (int d = 0; d < 100; d++) sms[d] = 100 + d;
  there = false;
  assert(qmm::kv_max_ctas(1) == 152 && qmm::kv_max_ctas(2) == 304);   // no device yet
  there = true;
  for (int pass = 0; pass < 2; pass++)
    for (device = 0; device < 100; device += 33) assert(qmm::kv_max_ctas(2) == 2 * (100 + device));
  assert(asked == 6);                                                // once a device, and each time past the 64 that are kept
  device = 33;
  assert(qmm::kv_max_ctas(10) == 1024);
  std::vector<std::thread> all;
  for (int t = 0; t < 8; t++)
    all.emplace_back([t] {
      for (int i = 0; i < 1000; i++) {
        device = (t + i) % 60;
        if (qmm::kv_max_ctas(1) != 100 + device) std::abort();
      }
    });
  for (auto &t : all) t.join();
  puts("ok");
}
"""


def test_grid_follows_the_device(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(SOURCE)
    cuda = os.path.join(os.path.dirname(os.path.dirname(qbuild.nvcc())) or "/usr/local/cuda", "include")
    subprocess.run(["g++", "-std=c++17", "-I", qbuild.CSRC, "-I", cuda, str(src), "-o", str(exe), "-pthread"], check=True)
    assert subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout == "ok\n"
