"""The widest vectors that the expert calls take: what the kernels' arguments
hold for them, read on the host (the kernels' own source, no launch)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include "kernels_moe.cu"

#include <cstdio>

namespace grs {
void set_last_error(const std::string&) {}
}

int main() {
  grs_moe s{3, 1, 0, 4, GRS_MAX_WIDTH, GRS_DTYPE_FP32, 0};
  const bool taken = grs::check_moe(&s, "") == GRS_OK;
  const auto copy = grs::moe_copy_args(&s, nullptr, nullptr, nullptr);
  const auto sum = grs::moe_args<float>(&s, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, true);
  // widths in elements (of the copy: 16-bit halves) and the last unit's first element
  printf("%d %lld %d %d %d\n", taken, (long long)copy.units * 8, (copy.units - 1) * 8, sum.d, (sum.units - 1) * 8);
}
"""


def test_the_widest_vectors_are_addressed_in_64_bits(tmp_path):
    from gradient_reduction_sharded_gb300 import _build
    src, exe = tmp_path / "widths.cu", tmp_path / "widths"
    src.write_text(SOURCE)
    try:
        nvcc = _build.nvcc()
    except RuntimeError:
        pytest.skip("no nvcc")
    subprocess.run([nvcc, "-std=c++17", "-O0", "-Xcicc", "-O0", "-Xptxas", "-O0", "-I", os.path.join(ROOT, "include"), "-I", _build.CSRC, *_build.ARCH,
                    str(src), "-o", str(exe)], check=True, capture_output=True, text=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    w = 1 << 30
    assert got == [1, 2 * w, 2 * w - 8, w, w - 8]
