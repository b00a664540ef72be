"""CPU: the parts that the gradient of layer normalization spreads its rows over,
from the host header: whatever the number of CTAs that a device holds at once, no
call uses more parts than its workspace has, and rows that are not whole vectors
keep their distance."""
import os
import subprocess

from residual_add_normalization_gb300 import buildlib

PROGRAM = r"""
#include <cstdio>
#include "layer.h"
using namespace b200norm;
int main() {
  long wrong = 0;
  for (int64_t rows : {1, 2, 3, 5, 7, 8, 9, 15, 16, 100, 152, 153, 500, 4096, 1 << 20})
    for (int64_t hidden : {128, 1027, 8195, 65535})
      for (int ve : {4, 8})
        for (int fit = 1; fit <= 1000; ++fit) {
          const int have = layer_grad_parts(rows, hidden);
          const int parts = window_parts(rows, have < fit ? have : fit, ve);
          if (parts < 1 || parts > rows || parts > have || (parts < rows && parts % ve)) {
            if (!wrong++) std::printf("rows %ld hidden %ld ve %d fit %d: %d of %d\n", (long)rows,
                                      (long)hidden, ve, fit, parts, have);
          }
        }
  if (!wrong) std::printf("ok\n");
  return wrong ? 1 : 0;
}
"""


def test_parts_stay_in_the_workspace(tmp_path):
    cuda = os.path.join(os.path.dirname(os.path.dirname(buildlib.nvcc())), "include")
    src, exe = tmp_path / "parts.cpp", tmp_path / "parts"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", f"-I{buildlib.CSRC}", f"-I{buildlib.INCLUDE}",
                    f"-I{cuda}", str(src), "-o", str(exe)], check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.stdout.strip() == "ok", r.stdout
