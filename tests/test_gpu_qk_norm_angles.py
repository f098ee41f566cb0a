"""Sines and cosines of the rotation as they enter results in fp32: with a head
of ones, no eps and a gradient of one in each pair, the weight's gradient is
the cosine and the sine itself."""
import math

import pytest
import torch

from operators_support import DT, binding, dtype_code, ptr, stream

pytestmark = pytest.mark.gpu

# The angle is a multiple of 2^-32 turn (off by half of that), then an fp32 number of half turns in [-1, 1] (2^-25 of a
# half turn at most); sine and cosine are off by at most two units of the binade below 1 (2^-24 each).
LIMIT = 2 * math.pi * 2.0 ** -33 + math.pi * 2.0 ** -25 + 2 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


# Heads of whole 16-byte chunks and others, both kinds of pairs.
@pytest.mark.parametrize("d, rot, pairs", [(128, 128, False), (128, 64, True), (20, 16, False), (22, 12, True)])
@pytest.mark.parametrize("act", ["bf16", "fp32"])
def test_angles_in_gradients_in_fp32(d, rot, pairs, act):
    grs, g = binding(), torch.Generator().manual_seed(d)
    inv = (torch.rand(rot // 2, generator=g, dtype=torch.float64) * 2 * math.pi).tolist()
    fractions = grs.grs_rope_turns(inv)
    turns = torch.tensor(fractions, dtype=torch.uint64, device="cuda")
    shape = grs.make_qk_norm(1, 1, 0, d, rot, 0.0, dtype_code(act), dtype_code("fp32"), dtype_code("fp32"), pairs)
    ws = torch.empty(max(16, grs.grs_qk_norm_workspace_bytes(shape)), dtype=torch.uint8, device="cuda")
    x = torch.ones(d, dtype=DT[act], device="cuda")
    first = range(0, rot, 2) if pairs else range(rot // 2)
    second = range(1, rot, 2) if pairs else range(rot // 2, rot)
    dy = torch.zeros(d, dtype=DT[act], device="cuda")
    dy[list(first)] = 1
    dw = torch.empty(d, device="cuda")
    worst = 0.0
    for position in torch.randint(-2 ** 31, 2 ** 31 - 1, (100,), generator=g).tolist() + [0, 1, -1, 7]:
        at = torch.tensor([position], dtype=torch.int32, device="cuda")
        grs.grs_qk_norm_backward(shape, ptr(dy), None, ptr(x), None, None, None, ptr(at), ptr(turns), None, None, ptr(dw), None, ptr(ws), stream())
        got = dw.double().cpu()
        for i, j, t in zip(first, second, fractions):
            angle = 2 * math.pi * ((position * t % 2 ** 64) / 2.0 ** 64)
            worst = max(worst, abs(float(got[i]) - math.cos(angle)), abs(float(got[j]) + math.sin(angle)))
    assert worst <= LIMIT, worst / LIMIT
