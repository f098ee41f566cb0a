"""How exact the list's norm is: pairs of floats, not floats.

An accumulator takes at most 36 squares between additions in 64 bits.  With
u = 2^-24, TwoSum's error terms are at most u of the sum each, and their own
additions add at most u of their sum: 36 * 37 / 2 * u^2 < 2^-38 of S; fp32
gradients add the squares' error terms, twice as many additions of twice as
much: 2^-36.  Plain fp32 sums are off by 2^-21 in the second test.
"""
import math

import numpy as np
import pytest
import torch

from test_gpu_list_adamw import List, grs  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [[1], [5, 255, 257], [2047, 2049, 7 * 2048 + 300], [100003, 31]]


def norm_of(grs, t, values, n_micro=1):
    """S of these fp32 values (rounded to the list's type), and what it is."""
    total = []
    for i, (buf, k, o) in enumerate(zip(t.store, t.numels, t.off)):
        x = torch.from_numpy(values[o:o + k].astype(np.float32)).to(buf.dtype)
        buf[t.shift:t.shift + k] = x.cuda()
        total.append(x.double().numpy())
    grs.grs_tensors_norm_sq(t.h, t.gp.data_ptr(), t.dt, n_micro, t.ws.data_ptr(), t.norm.data_ptr(), t.stream())
    x = np.concatenate(total)
    return float(t.norm.cpu()[0]), math.fsum((x * x).tolist()) / n_micro ** 2


@pytest.mark.parametrize("numels", SHAPES)
@pytest.mark.parametrize("bf16,shift", [(False, 0), (True, 0), (True, 1), (False, 3), (True, 5)])
@pytest.mark.parametrize("kind", ["normal", "wide", "large", "small"])
def test_s_to_36_bits(grs, numels, bf16, shift, kind):  # noqa: F811
    t = List(grs, numels, bf16, shift, seed=31)
    rng = np.random.default_rng(32)
    x = rng.standard_normal(t.n)
    if kind == "wide":
        x *= np.exp2(rng.uniform(-20, 20, t.n))
    elif kind == "large":
        x = np.clip(x, -4, 4) * 2.0 ** 58
    elif kind == "small":
        x = np.copysign(np.maximum(np.abs(x), 2.0 ** -8), x) * 2.0 ** -43
    got, want = norm_of(grs, t, x, 4)
    assert abs(got - want) <= 2.0 ** -36 * want, abs(got / want - 1)
    assert grs.grs_tensors_check_device_errors(t.h, t.stream()) == grs.GRS_OK
    t.close()


@pytest.mark.parametrize("bf16,shift", [(False, 0), (True, 0), (True, 3)])
def test_small_numbers_behind_large_ones_count(grs, bf16, shift):  # noqa: F811
    """The first 256 elements of each tile of 2048 are 1, each other's square is lost when it is added to theirs in fp32."""
    t = List(grs, [40 * 2048], bf16, shift, seed=33)
    x = np.full(t.n, 1.203125 * 2.0 ** -12)
    x.reshape(-1, 2048)[:, :256] = 1
    got, want = norm_of(grs, t, x)
    assert abs(got - want) <= 2.0 ** -36 * want, abs(got / want - 1)
    t.close()
