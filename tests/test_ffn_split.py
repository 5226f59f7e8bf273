"""The cut of a sum's steps into parts (csrc/ffn_split.h), compiled for the host: the parts cover every
step once, in order and evenly, for sums of up to 2^31 rows (2^25 steps) and up to 256 parts."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

PROGRAM = r"""
#include <cstdio>
#include "ffn_split.h"
int main() {
  const uint32_t steps[] = {0, 1, 2, 7, 8, 31, 255, 256, 257, 1000, 4095, 65535, 65536, 65537, 1000003, (1u << 24) - 1,
                            1u << 24, (1u << 24) + 1, 20000001, (1u << 25) - 1, 1u << 25};
  for (uint32_t n : steps)
    for (uint32_t parts = 1; parts <= 256; parts++) {
      if (glu::part_begin(n, 0, parts) != 0 || glu::part_begin(n, parts, parts) != n) return printf("%u %u\n", n, parts), 1;
      for (uint32_t p = 0; p < parts; p++) {
        const uint32_t a = glu::part_begin(n, p, parts), b = glu::part_begin(n, p + 1, parts);
        const uint64_t want = (uint64_t)n * p / parts;
        if (a != want || b < a || b - a < n / parts || b - a > n / parts + 1)
          return printf("%u steps, part %u of %u: %u .. %u\n", n, p, parts, a, b), 1;
      }
    }
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_parts_cover_every_step_once(tmp_path):
    src, exe = tmp_path / "split.cpp", tmp_path / "split"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-I",
                    os.path.join(ROOT, "glu_activation_microscaling_amd", "csrc"), str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
