"""The copies of int4_product's scales and zero points (csrc/blocks.h), restated
on the CPU: whatever byte a matrix starts at, no 16-byte block that is copied
reaches out of it, and every entry is copied."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "draft_verification_gb300", "csrc")

PROGRAM = r"""
#include <algorithm>
#include <cstdio>
#include "blocks.h"

// every stage of a matrix of `rows` rows, as int4_product_kernel copies them: `per` rows a stage
static bool check(uint64_t base, int entry, int V, long long ld, int rows, int per) {
  const uint64_t hi = base + ((rows - 1) * ld + V) * entry;
  const bool ragged = (base | hi) & 15;
  for (int v0 = 0; v0 < V; v0 += 128)
    for (int g = 0; g < rows; ++g) {
      const int g0 = g / per * per;
      const unsigned bytes = std::min(128, V - v0) * entry;
      const uint64_t src = base + (g * ld + v0) * entry, first = src & ~15ull;
      const unsigned lead = src - first;
      sv::Blocks b{0, (lead + bytes + 15) & ~15u};
      if (ragged && sv::blocks_may_stick_out(V, v0, g0 == 0, rows - g0 <= per))
        b = sv::blocks_within(src, bytes, base, hi);
      if (b.begin % 16 || b.end % 16 || b.begin > b.end || b.end > 272) return false;
      if (b.end > b.begin && (first + b.begin < base || first + b.end > hi)) return false;
      // less than a block is left to single bytes at either end
      if (b.end > b.begin && (b.begin > 16 || b.end + 16 < lead + bytes)) return false;
    }
  return true;
}

int main() {
  const int widths[] = {1, 2, 7, 8, 9, 15, 16, 17, 31, 100, 112, 113, 127, 128, 129, 136, 143, 144, 145, 255, 256, 257, 300, 384, 385, 500};
  for (int entry = 1; entry <= 2; ++entry)
    for (int at = 0; at < 16; at += entry)
      for (int V : widths)
        for (int pad : {0, 1, 3, 8, 15, 16, 40})
          for (int rows : {1, 2, 3, 4, 5, 8, 9, 17})
            for (int per : {2, 4, 8})
              if (!check(0x10000 + at, entry, V, V + pad, rows, per))
                return std::printf("entry %d at %d V %d pad %d rows %d per %d\n", entry, at, V, pad, rows, per), 1;
  return 0;
}
"""


def test_no_copied_block_reaches_out_of_the_matrix(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "blocks.cpp", tmp_path / "blocks"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout
