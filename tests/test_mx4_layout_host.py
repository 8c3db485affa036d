"""What a CTA of the microscaled product holds in shared memory, for every number of experts and parts of K, and quotients by
sizes: their header compiled for the host."""
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


DIVISOR = r"""
#include <cassert>
#include <cstdio>
#include <vector>
#include "mx4_layout.h"

int main() {
  const uint32_t most = 0x7FFFFFFFu;
  std::vector<uint32_t> sizes;
  for (uint32_t d = 1; d <= 3000; d++) sizes.push_back(d);
  for (int bit = 11; bit < 31; bit++)
    for (int off = -2; off <= 2; off++) sizes.push_back((1u << bit) + off), sizes.push_back(3 * (1u << (bit - 1)) + off);
  for (uint32_t off = 0; off < 5; off++) sizes.push_back(most - off);
  uint32_t seed = 1;
  for (int i = 0; i < 20000; i++) sizes.push_back((seed = seed * 1664525u + 1013904223u) % most + 1);
  for (uint32_t d : sizes) {
    const qmm::Divisor by(d);
    auto check = [&](uint64_t n) {
      if (n > most) return;
      uint32_t r = (uint32_t)n;
      assert(by.quotient(r) == r / d && by.split(r) == n / d && r == n % d);
    };
    for (uint64_t n = 0; n < 40; n++) check(n), check(most - n);
    for (uint64_t q : {(uint64_t)1, (uint64_t)2, (uint64_t)7, (uint64_t)most / d, (uint64_t)most / d / 2, (uint64_t)most / d / 3})
      for (int off = -2; off <= 2; off++)
        if ((int64_t)(q * d) + off >= 0) check(q * d + off);
    for (int i = 0; i < 20; i++) check((seed = seed * 1664525u + 1013904223u) >> 1);
  }
  puts("ok");
}
"""


def test_shared_memory(tmp_path):
    run(tmp_path, SOURCE)


def test_quotients(tmp_path):
    run(tmp_path, DIVISOR)


def run(tmp_path, source):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(source)
    cuda = os.path.join(os.path.dirname(os.path.dirname(qbuild.nvcc())) or "/usr/local/cuda", "include")
    subprocess.run(["g++", "-std=c++17", "-I", qbuild.CSRC, "-I", cuda, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout == "ok\n"
