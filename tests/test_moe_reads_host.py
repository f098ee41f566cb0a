"""What the expert kernels read of a vector that starts anywhere: nothing
behind it and nothing before the matrix, so that a matrix of exactly a rank's
rows is enough.  The kernels' own chunk rule, walked on the host."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include <cstdio>
#include <vector>
#include "shifted.cuh"

// Every vector of a matrix of `rows` vectors of d elements whose first lies `start` elements after a 16-byte boundary.
static int walk(int el, int d, int rows, int start) {
  int bad = 0;
  for (int v = 0; v < rows; ++v)
    for (int run = 0; run < d; run += 256) {
      std::vector<char> read(size_t(rows) * d + 1024, 0);
      const int off = (start + v * d + run) % el;  // the same for every lane: 8 elements are whole chunks
      for (int lane = 0; lane < 32; ++lane)
        for (int i = 0; i <= 8 / el; ++i) {
          if (i == 8 / el && !(off != 0 && lane == 31)) continue;  // the chunk behind the warp's last lane
          const int c = run + lane * 8;
          const grs::Span s = grs::chunk_span(el, i, off, v * d + c < 8 ? v * d + c : 8, d - c);
          for (int q = s.lo < 0 ? 0 : s.lo; q < (s.hi < el ? s.hi : el); ++q) {
            const long at = long(v) * d + c - off + i * el + q;
            if (at < 0 || at >= long(v + 1) * d) ++bad;
            else read[at] = 1;
          }
        }
      for (int e = run; e < d && e < run + 256; ++e) bad += !read[size_t(v) * d + e];  // all that is needed
    }
  return bad;
}

int main() {
  const int widths[] = {1, 3, 7, 8, 12, 31, 33, 67, 255, 256, 257, 260, 263, 264, 300, 515, 1027, 2051, 2052};
  for (int el : {8, 4})
    for (int d : widths)
      for (int rows : {1, 2, 5})
        for (int start = 0; start < el; ++start)
          if (int bad = walk(el, d, rows, start)) printf("el %d d %d rows %d start %d: %d\n", el, d, rows, start, bad);
  printf("walked\n");
}
"""


def test_a_vector_is_read_to_its_end_and_no_further(tmp_path):
    from gradient_reduction_sharded_gb300 import _build
    src, exe = tmp_path / "walk.cu", tmp_path / "walk"
    src.write_text(SOURCE)
    try:
        nvcc = _build.nvcc()
    except RuntimeError:
        pytest.skip("no nvcc")
    subprocess.run([nvcc, "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", _build.CSRC, *_build.ARCH, str(src), "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    assert subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout == "walked\n"
