"""A block of the experts' products gives up (through the self-test), as if a
wait had lasted too long: the call ends, the flag is reported once, nothing
outside the outputs is touched and the next call is as ever."""
import pytest
import torch

from operators_support import DT, binding, ptr, stream
from test_gpu_experts import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def inside(shape, dtype):
    """A tensor with 512 elements of 7 before and behind it, and whether these are as they were."""
    n = torch.Size(shape).numel()
    whole = torch.full((n + 1024,), 7.0, dtype=dtype, device="cuda")
    return whole[512:512 + n].view(shape), lambda: bool((whole[:512] == 7).all()) and bool((whole[512 + n:] == 7).all())


def quit_at(c, quitter, tile, rows=True, weights=True):
    dxs, dxs_kept = inside((c.rows, c.k), DT[c.act])
    dw, dw_kept = inside(c.w.shape, DT[c.grad])
    binding().grs_selftest_experts_wait(c.shape, ptr(c.dys), ptr(c.xs), ptr(c.w), ptr(c.offsets), ptr(dxs) if rows else None,
                                        ptr(dw) if weights else None, ptr(c.ws), quitter, tile, stream())
    torch.cuda.synchronize()
    assert dxs_kept() and dw_kept()
    return dxs, dw


# Rows in tiles of 16, 64, 128 and (two blocks) 256, weights in small and (two blocks) large ones, several sections, slices.
CASES = [([10, 6], 264, 136, "bf16"), ([40, 20], 264, 136, "bf16"), ([100, 90], 264, 136, "fp32"), ([500] * 4, 2560, 520, "bf16"), ([500] * 4, 2560, 520, "fp32"),
         ([4500, 600], 2560, 1032, "bf16"), ([700], 16384, 8, "bf16")]


@pytest.mark.parametrize("counts, k, n, grad", CASES)
@pytest.mark.parametrize("quitter, tile", [(0, 0), (1, 0), (0, 1)])
def test_a_call_that_gives_up_ends(counts, k, n, grad, quitter, tile):
    grs = binding()
    c = Case(counts, k, n, "bf16", grad)
    want = c.backward()
    assert grs.grs_operators_check_device_errors(stream()) == grs.GRS_OK
    for rows, weights in ((True, False), (False, True)):
        quit_at(c, quitter, tile, rows, weights)
        status = grs.grs_operators_check_device_errors(stream())
        # (a block may have had no second tile)
        assert status == grs.GRS_ERR_TIMEOUT or (tile > 0 and status == grs.GRS_OK)
        assert grs.grs_operators_check_device_errors(stream()) == grs.GRS_OK
        again = c.backward()
        assert grs.grs_operators_check_device_errors(stream()) == grs.GRS_OK
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


def test_a_block_that_the_call_does_not_have_gives_up_nothing():
    grs = binding()
    c = Case([40, 20], 264, 136)
    want = c.backward()
    got = quit_at(c, 100000, 0)
    assert grs.grs_operators_check_device_errors(stream()) == grs.GRS_OK
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_the_report_says_what_and_comes_once_from_any_stream():
    grs = binding()
    c = Case([40, 20], 264, 136)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        quit_at(c, 0, 0)
    assert grs.grs_operators_check_device_errors(stream()) == grs.GRS_ERR_TIMEOUT
    assert "timed out" in grs.grs_last_error()
    assert grs.grs_operators_check_device_errors(side.cuda_stream) == grs.GRS_OK
