"""The header says which kernels a checked build checks; the sources agree."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_header_names_the_kernels_without_checks():
    with open(os.path.join(ROOT, "include", "grs.h")) as f:
        header = re.sub(r"[\s*]+", " ", f.read())
    without = set()
    for path in glob.glob(os.path.join(ROOT, "gradient_reduction_sharded_gb300", "csrc", "*.cu")):
        with open(path) as f:
            src = f.read()
        if "__global__" in src and "GRS_CHECK(" not in src:
            without.add(os.path.basename(path))
    assert without == {"kernels_layernorm.cu", "kernels_moe.cu"}
    assert "every kernel checks each index" not in header
    assert "The kernels of grs_layernorm_ and grs_moe_ have no such checks" in header
