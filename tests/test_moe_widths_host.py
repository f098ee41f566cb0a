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


WHOLE = r"""
#include "kernels_moe.cu"

#include <cstdio>

namespace grs {
void set_last_error(const std::string&) {}
}

int main() {
  void* at[2] = {reinterpret_cast<void*>(uintptr_t(4096)), reinterpret_cast<void*>(uintptr_t(4096 + 8))};
  for (int dtype : {GRS_DTYPE_BF16, GRS_DTYPE_FP32})
    for (int hidden : {8, 12, 2048, 2052, 2056, 2051})
      for (void* p : at) {
        const grs_moe s{3, 1, 0, 4, hidden, dtype, 0};
        printf("%d", grs::moe_whole(&s, p, nullptr, at[0]));
      }
  printf("\n");
}
"""


def test_the_fast_path_is_what_the_header_says(tmp_path):
    """16-byte aligned vectors of a multiple of 8 elements, in either type."""
    import re

    from gradient_reduction_sharded_gb300 import _build
    src, exe = tmp_path / "whole.cu", tmp_path / "whole"
    src.write_text(WHOLE)
    try:
        nvcc = _build.nvcc()
    except RuntimeError:
        pytest.skip("no nvcc")
    subprocess.run([nvcc, "-std=c++17", "-O0", "-Xcicc", "-O0", "-Xptxas", "-O0", "-I", os.path.join(ROOT, "include"), "-I", _build.CSRC, *_build.ARCH,
                    str(src), "-o", str(exe)], check=True, capture_output=True, text=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.strip()
    assert got == "".join("10" if h % 8 == 0 else "00" for h in (8, 12, 2048, 2052, 2056, 2051)) * 2
    with open(os.path.join(ROOT, "include", "grs.h")) as f:
        header = re.sub(r"[\s*]+", " ", f.read())
    assert "16 bytes, with hidden a multiple of 8, is fastest in either type" in header
