"""Host side of the experts' products, the embedding and the query and key
norms: struct layouts, refusals (before anything is launched), the rotation's
frequencies."""
import ctypes
import math
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def grs():
    from gradient_reduction_sharded_gb300 import _build
    _build.build()
    from gradient_reduction_sharded_gb300 import grs as g
    return g


def test_struct_layouts_match_the_c_compiler(grs, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    names = ("grs_experts", "grs_embedding", "grs_qk_norm")
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


def refused(grs, status, call, *args):
    with pytest.raises(grs.GrsError) as e:
        call(*args)
    assert e.value.status == status, e.value


# Addresses that no call may reach: every one of these is refused on the host.
A = 1 << 20


@pytest.mark.parametrize("status, change", [
    ("SHAPE", {"rows": -1}), ("SHAPE", {"rows": (1 << 31) - (1 << 16) + 1}), ("SHAPE", {"experts": 0}), ("SHAPE", {"experts": 1025}),
    ("SHAPE", {"in_features": 0}), ("SHAPE", {"out_features": 0}), ("SHAPE", {"in_features": (1 << 30) + 1}),
    ("SHAPE", {"ld_x": 15}), ("SHAPE", {"ld_y": 7}), ("SHAPE", {"ld_x": -16}), ("SHAPE", {"ld_y": (1 << 30) + 1}),
    ("INVALID_ARG", {"dtype": 2}), ("INVALID_ARG", {"grad_dtype": -1})])
def test_experts_refuse_shapes(grs, status, change):
    s = grs.make_experts(10, 3, 16, 8, grs.GRS_DTYPE_BF16, grs.GRS_DTYPE_FP32)
    for k, v in change.items():
        setattr(s, k, v)
    st = getattr(grs, "GRS_ERR_" + status)
    refused(grs, grs.GRS_ERR_INVALID_ARG, grs.grs_experts_workspace_bytes, s)
    refused(grs, st, grs.grs_experts_forward, s, A, A, A, A, A, 0)
    refused(grs, st, grs.grs_experts_backward, s, A, A, A, A, A, A, A, 0)


def test_experts_refuse_pointers(grs):
    s = grs.make_experts(10, 3, 16, 8, grs.GRS_DTYPE_BF16, grs.GRS_DTYPE_FP32)
    for i in range(4):
        args = [A] * 5
        args[i] = None
        refused(grs, grs.GRS_ERR_INVALID_ARG, grs.grs_experts_forward, s, *args, 0)
    for i, off in ((0, 2), (1, 8), (2, 2), (3, 1), (4, 8)):
        args = [A] * 5
        args[i] += off
        refused(grs, grs.GRS_ERR_ALIGNMENT, grs.grs_experts_forward, s, *args, 0)
    refused(grs, grs.GRS_ERR_INVALID_ARG, grs.grs_experts_backward, s, None, A, A, A, A, A, A, 0)
    refused(grs, grs.GRS_ERR_INVALID_ARG, grs.grs_experts_backward, s, A, None, A, A, None, A, A, 0)
    refused(grs, grs.GRS_ERR_INVALID_ARG, grs.grs_experts_backward, s, A, A, None, A, A, None, A, 0)
    refused(grs, grs.GRS_ERR_INVALID_ARG, grs.grs_experts_backward, s, A, A, A, None, A, A, A, 0)
    for i, off in ((0, 8), (1, 2), (2, 4), (3, 2), (4, 1), (5, 2), (6, 4)):
        args = [A] * 7
        args[i] += off
        refused(grs, grs.GRS_ERR_ALIGNMENT, grs.grs_experts_backward, s, *args, 0)
    grs.grs_experts_forward(grs.make_experts(0, 3, 16, 8, 0, 1), None, None, None, None, None, 0)  # no rows: nothing to do
    grs.grs_experts_backward(grs.make_experts(0, 3, 16, 8, 0, 1), None, None, None, None, None, None, None, 0)


@pytest.mark.parametrize("status, change", [
    ("SHAPE", {"tokens": -1}), ("SHAPE", {"tokens": (1 << 31) - (1 << 16) + 1}), ("SHAPE", {"hidden": 0}), ("SHAPE", {"hidden": (1 << 30) + 1}),
    ("INVALID_ARG", {"row_begin": -1}), ("INVALID_ARG", {"row_end": 4}), ("INVALID_ARG", {"dtype": 3}), ("INVALID_ARG", {"grad_dtype": 2})])
def test_embedding_refuses_shapes(grs, status, change):
    s = grs.make_embedding(5, 4, 20, 16, 1.0, grs.GRS_DTYPE_FP32, grs.GRS_DTYPE_BF16)
    for k, v in change.items():
        setattr(s, k, v)
    st = getattr(grs, "GRS_ERR_" + status)
    refused(grs, grs.GRS_ERR_INVALID_ARG, grs.grs_embedding_workspace_bytes, s)
    refused(grs, st, grs.grs_embedding_forward, s, A, A, A, 0)
    refused(grs, st, grs.grs_embedding_backward, s, A, A, A, A, 0)


def test_embedding_refuses_pointers(grs):
    s = grs.make_embedding(5, 4, 20, 16, 1.0, grs.GRS_DTYPE_FP32, grs.GRS_DTYPE_BF16)
    for i in range(3):
        refused(grs, grs.GRS_ERR_INVALID_ARG, grs.grs_embedding_forward, s, *[None if j == i else A for j in range(3)], 0)
        refused(grs, grs.GRS_ERR_ALIGNMENT, grs.grs_embedding_forward, s, *[A + 2 if j == i else A for j in range(3)], 0)
    for i, off in enumerate((2, 2, 1, 8)):
        refused(grs, grs.GRS_ERR_INVALID_ARG, grs.grs_embedding_backward, s, *[None if j == i else A for j in range(4)], 0)
        refused(grs, grs.GRS_ERR_ALIGNMENT, grs.grs_embedding_backward, s, *[A + off if j == i else A for j in range(4)], 0)
    grs.grs_embedding_forward(grs.make_embedding(0, 0, 1, 1, 1.0, 0, 0), None, None, None, 0)


@pytest.mark.parametrize("status, change", [
    ("SHAPE", {"tokens": -1}), ("SHAPE", {"q_heads": -1}), ("SHAPE", {"k_heads": -1}), ("SHAPE", {"head_dim": 0}),
    ("SHAPE", {"head_dim": 1025}), ("SHAPE", {"q_heads": 1 << 30}), ("SHAPE", {"rotary_dim": 3}), ("SHAPE", {"rotary_dim": 18}),
    ("SHAPE", {"rotary_dim": -2}), ("SHAPE", {"ld_q": 31}), ("SHAPE", {"ld_k": 1}), ("SHAPE", {"ld_qo": 5}), ("SHAPE", {"ld_ko": -1}),
    ("INVALID_ARG", {"interleaved": 2}), ("INVALID_ARG", {"eps": -1.0}), ("INVALID_ARG", {"eps": math.nan}),
    ("INVALID_ARG", {"dtype": 2}), ("INVALID_ARG", {"param_dtype": 2}), ("INVALID_ARG", {"grad_dtype": 2})])
def test_qk_norm_refuses_shapes(grs, status, change):
    s = grs.make_qk_norm(3, 2, 1, 16, 8, 1e-6, 0, 0, 0)
    for k, v in change.items():
        setattr(s, k, v)
    st = getattr(grs, "GRS_ERR_" + status)
    refused(grs, grs.GRS_ERR_INVALID_ARG, grs.grs_qk_norm_workspace_bytes, s)
    refused(grs, st, grs.grs_qk_norm_forward, s, *[A] * 8, 0)
    refused(grs, st, grs.grs_qk_norm_backward, s, *[A] * 13, 0)


def test_qk_norm_refuses_pointers(grs):
    s = grs.make_qk_norm(3, 2, 1, 16, 8, 1e-6, 0, 0, 0)
    # q, k, wq, wk, positions, turns, qo, ko
    far = [A + 4096 * i for i in range(13)]
    for i in (0, 1, 4, 5, 6, 7):
        refused(grs, grs.GRS_ERR_INVALID_ARG, grs.grs_qk_norm_forward, s, *[None if j == i else far[j] for j in range(8)], 0)
    for i, off in enumerate((1, 1, 1, 1, 2, 4, 1, 1)):
        refused(grs, grs.GRS_ERR_ALIGNMENT, grs.grs_qk_norm_forward, s, *[far[j] + off * (j == i) for j in range(8)], 0)
    # dqo, dko, q, k, wq, wk, positions, turns, dq, dk, dwq, dwk, workspace
    for i in (0, 1, 2, 3, 6, 7, 12):
        refused(grs, grs.GRS_ERR_INVALID_ARG, grs.grs_qk_norm_backward, s, *[None if j == i else far[j] for j in range(13)], 0)
    for i, off in enumerate((1, 1, 1, 1, 1, 1, 2, 4, 1, 1, 1, 1, 8)):
        refused(grs, grs.GRS_ERR_ALIGNMENT, grs.grs_qk_norm_backward, s, *[far[j] + off * (j == i) for j in range(13)], 0)
    # In place only with one distance of tokens.
    s.ld_q = 64
    refused(grs, grs.GRS_ERR_INVALID_ARG, grs.grs_qk_norm_forward, s, *far[:6], far[0], far[7], 0)
    refused(grs, grs.GRS_ERR_INVALID_ARG, grs.grs_qk_norm_backward, s, *far[:8], far[0], *far[9:], 0)


def test_turns_are_the_frequencies_modulo_a_turn(grs):
    rng = random.Random(5)
    freqs = [1.0, 0.0, -1.0, 2 * math.pi, -2 * math.pi, 1e6 ** (-126 / 128), 1e-300, 6.5, 1e9, -1e-30] + [10 ** rng.uniform(-12, 3) * rng.choice((-1, 1)) for _ in range(100)]
    for f, t in zip(freqs, grs.grs_rope_turns(freqs)):
        whole = f / (2 * math.pi)
        off = (t / 2 ** 64 - whole) % 1.0
        # the quotient's rounding (and the constant's), the difference's, 2^-64 of the whole turn
        assert min(off, 1 - off) <= abs(whole) * 2 ** -52 + 2 ** -53, (f, t)
    for bad in (math.inf, -math.inf, math.nan):
        refused(grs, grs.GRS_ERR_INVALID_ARG, grs.grs_rope_turns, [1.0, bad])
    assert grs.grs_rope_turns([]) == []
