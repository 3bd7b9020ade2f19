"""Where the matrix-vector kernel reads codes, checked on the CPU: the header's
arithmetic is compiled for the host and tried for every chunk of many row lengths."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "grouped_nf4_gemm_quantize_amd", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "matvec_index.h"
using namespace nf4moe;
int main() {
  for (int K = 32; K <= 20480; K += 32) {
    const int bytes = K / 2, chunks = (K + kMvChunk - 1) / kMvChunk;
    for (int c = 0; c < chunks; ++c)
      for (int q = 0; q < 4; ++q) {
        const int at = mv_code_byte(c, q, bytes), want = c * (kMvChunk / 2) + 16 * q;
        // inside the row, aligned, and the lane's own bytes wherever the row has them
        if (at < 0 || at + 16 > bytes || at % 16 || (want < bytes && at != want)) {
          std::printf("K=%d chunk=%d quarter=%d reads bytes %d..%d of %d\n", K, c, q, at, at + 15,
                      bytes);
          return 1;
        }
      }
  }
  return 0;
}
"""


def test_code_reads_stay_in_their_row(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "index.cpp", tmp_path / "index"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout
