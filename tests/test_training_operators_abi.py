"""The training operators' structs agree with the C compiler, and the checked
build's list kernels find no index out of place (on the GPU)."""
import ctypes
import os
import re
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_struct_layouts_match_the_c_compiler(tmp_path):
    from gradient_reduction_sharded_gb300 import _build
    _build.build()
    from gradient_reduction_sharded_gb300 import grs
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    names = ("grs_tensors_info", "grs_norm", "grs_moe")
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "grs.h"', "int main(void) {"]
    for s in names:
        lines.append(f'  printf("{s} sizeof %zu\\n", sizeof({s}));')
        for field, _ in getattr(grs, s)._fields_:
            lines.append(f'  printf("{s} {field} %zu\\n", offsetof({s}, {field}));')
    lines += ["  return 0;", "}"]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines) + "\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    got = {(s, f): int(v) for s, f, v in (line.split() for line in out.splitlines())}
    for s in names:
        cls = getattr(grs, s)
        assert got[(s, "sizeof")] == ctypes.sizeof(cls)
        for field, _ in cls._fields_:
            assert got[(s, field)] == getattr(cls, field).offset, (s, field)


@pytest.mark.gpu
def test_list_suite_passes_on_the_checked_build():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from gradient_reduction_sharded_gb300 import _build
    lib = _build.build_checked()
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", "-m", "gpu",
                        "tests/test_gpu_list_adamw.py"], cwd=ROOT, env=dict(os.environ, GRS_LIBRARY=lib), capture_output=True,
                       text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    m = re.search(r"(\d+) passed", r.stdout)
    assert m and int(m.group(1)) >= 50, r.stdout[-2000:]
