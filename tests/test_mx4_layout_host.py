"""What a CTA of the microscaled product holds in shared memory, for every number of experts and parts of K: its header compiled
for the host."""
import os
import subprocess

from quantized_weight_gb300 import build as qbuild

SOURCE = r"""
#include <cassert>
#include <cstdio>
#include "mx4_layout.h"

using namespace qmm::mx4;

int main() {
  // an SM of compute capability 10.3: 228 KB of shared memory, 227 a CTA, handed out by 128 bytes with 1 KB more a CTA
  const int sm = 228 * 1024, most = 227 * 1024, kept = 1024, unit = 128;
  for (int experts = 1; experts <= 1024; experts++)
    for (int split = 1; split <= MAX_SPLIT; split *= 2) {
      const int n = ring_stages(false, 64, 1, split, experts, true);
      assert(n >= 2 && n <= MAX_STAGES);
      const int total = (layout(false, 64, 1, n, split, experts).total + unit - 1) / unit * unit;
      assert(2 * (total + kept) <= sm);                                                    // two CTAs do fit an SM
      assert(2 * (total + layout(false, 64, 1, n, split, experts).stage + kept) > sm);     // with as deep a ring as they can
    }
  const struct { bool gated; int ts, ctas, parts; } one[] = {{false, 64, 1, 8}, {false, 128, 1, 1}, {false, 192, 1, 1}, {false, 256, 1, 1},
      {false, 256, 2, 1}, {true, 64, 1, 4}, {true, 128, 1, 1}, {true, 128, 2, 1}};
  for (const auto &k : one)
    for (int experts = 1; experts <= 1024; experts++)
      for (int split = 1; split <= k.parts; split *= 2) {
        const int n = ring_stages(k.gated, k.ts, k.ctas, split, experts, false);
        assert(n >= 2 && n <= MAX_STAGES);
        assert(layout(k.gated, k.ts, k.ctas, n, split, experts).total <= most);
      }
  puts("ok");
}
"""


def test_shared_memory(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(SOURCE)
    cuda = os.path.join(os.path.dirname(os.path.dirname(qbuild.nvcc())) or "/usr/local/cuda", "include")
    subprocess.run(["g++", "-std=c++17", "-I", qbuild.CSRC, "-I", cuda, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout == "ok\n"
