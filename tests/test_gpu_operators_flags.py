"""A flag that a kernel raises while another thread reads and clears the flags
is reported by one of the two: every call that gives up is followed by a report,
whoever made it."""
import threading

import pytest
import torch

from operators_support import binding, ptr
from test_gpu_experts import Case

pytestmark = pytest.mark.gpu

CALLS = 1500


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def test_no_report_is_lost_between_two_that_look():
    grs = binding()
    c = Case([40, 20], 264, 136)
    dxs = torch.empty(c.rows, c.k, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    assert grs.grs_operators_check_device_errors(0) == grs.GRS_OK
    other, mine = torch.cuda.Stream().cuda_stream, torch.cuda.Stream().cuda_stream
    looks, found, end = [0], [0], threading.Event()

    def look():
        while not end.is_set():
            status = grs.grs_operators_check_device_errors(other)
            found[0] += status == grs.GRS_ERR_TIMEOUT
            looks[0] += 1

    thread = threading.Thread(target=look)
    thread.start()
    lost = 0
    try:
        for _ in range(CALLS):
            before = found[0]
            grs.grs_selftest_experts_wait(c.shape, ptr(c.dys), None, ptr(c.w), ptr(c.offsets), ptr(dxs), None, ptr(c.ws), 0, 0, mine)
            own = grs.grs_operators_check_device_errors(mine)  # (after the call's end)
            now = looks[0]
            while looks[0] < now + 2:  # a look that had begun has ended
                pass
            lost += own != grs.GRS_ERR_TIMEOUT and found[0] == before
    finally:
        end.set()
        thread.join()
    assert lost == 0
