"""A block of those that share wide rows gives up its wait for the others'
sums (with a short limit, through the self-test): what is finite in dx is
right, the rest is NaN, and the next call is as ever."""
import pytest
import torch

from test_gpu_layernorm import Case, check, grs  # noqa: F401
from test_gpu_layernorm_wide import gradients64

pytestmark = pytest.mark.gpu


def quit_at(c, act, par, limit_ns, quitter, row, dx=True):
    g = c.grs
    dt = {"bf16": g.GRS_DTYPE_BF16, "fp32": g.GRS_DTYPE_FP32}
    shape = g.make_norm(c.rows, c.cols, c.eps, dt[act], dt[par], g.GRS_DTYPE_FP32)
    gx = torch.full((c.rows, c.cols), 7.0, dtype=c.x.dtype, device="cuda")
    gw, gb = torch.zeros(c.cols, device="cuda"), torch.zeros(c.cols, device="cuda")
    g.grs_selftest_layernorm_wait(shape, c.dy.data_ptr(), c.x.data_ptr(), c.w.data_ptr(), c.mean.data_ptr(), c.rstd.data_ptr(),
                                  gx.data_ptr() if dx else None, gw.data_ptr(), gb.data_ptr(), c.ws.data_ptr(), limit_ns, quitter, row,
                                  torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    return gx, gw, gb


@pytest.mark.parametrize("act,cols,rows,quitter,row", [("bf16", 8200, 400, 1, 2), ("bf16", 16384, 400, 0, 0), ("fp32", 4104, 1500, 1, 1), ("fp32", 16384, 500, 2, 3),
                                                       ("bf16", 65536, 130, 7, 4), ("bf16", 20000, 10, 3, 0), ("fp32", 32768, 200, 5, 100)])
def test_a_lost_wait_leaves_nan_and_nothing_wrong(grs, act, cols, rows, quitter, row):  # noqa: F811
    c = Case(grs, rows, cols, act, act, "fp32", seed=cols)
    c.forward()
    gx, gw, gb = quit_at(c, act, act, 2_000_000, quitter, row)
    want = gradients64(c)
    for got, (w64, bound), what in zip((gw, gb), want[1:], ("dw", "db")):
        check(got, w64, bound, what)
    full = c.backward()[0]
    lost = torch.isnan(gx)
    status = grs.grs_layernorm_check_device_errors(torch.cuda.current_stream().cuda_stream)
    assert status == (grs.GRS_ERR_TIMEOUT if lost.any() else grs.GRS_OK)
    assert torch.equal(gx[~lost], full[~lost])  # right wherever it is a number
    # A cluster has every n-th row.  Its rows before the lost one are whole, of that one the block's columns are lost, then all.
    share = lost.float().mean(1)
    part = torch.nonzero((share > 0) & (share < 1))[:, 0]
    if len(part) == 0:
        assert not lost.any() and row > 0  # no cluster has as many rows
    else:
        first = int(part[0])
        n = first // row if row else len(part)
        assert first == row * n and part.tolist() == list(range(first, min(first + n, rows)))
        assert (share[:first] == 0).all() and (share[first + len(part):] == 1).all()
    assert torch.equal(c.backward()[0], full)
    check(full, *want[0], "dx")


def test_a_lost_wait_is_reported(grs):  # noqa: F811
    """Once, to the first check after it, also where it was on another stream; the calls that go well report nothing."""
    c = Case(grs, 100, 16384, "bf16", "bf16", "fp32", seed=5)
    c.forward()
    st = torch.cuda.current_stream().cuda_stream
    c.backward()
    assert grs.grs_layernorm_check_device_errors(st) == grs.GRS_OK
    quit_at(c, "bf16", "bf16", 2_000_000, 1, 0)
    assert grs.grs_layernorm_check_device_errors(st) == grs.GRS_ERR_TIMEOUT
    assert "timed out" in grs.grs_last_error()
    assert grs.grs_layernorm_check_device_errors(st) == grs.GRS_OK
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        quit_at(c, "bf16", "bf16", 2_000_000, 0, 0)
    assert grs.grs_layernorm_check_device_errors(side.cuda_stream) == grs.GRS_ERR_TIMEOUT
    c.backward()
    assert grs.grs_layernorm_check_device_errors(st) == grs.GRS_OK


def test_refusals(grs):  # noqa: F811
    c = Case(grs, 20, 8200, "bf16", "bf16", "fp32")
    c.forward()
    inv, sh = grs.GRS_ERR_INVALID_ARG, grs.GRS_ERR_SHAPE
    narrow = Case(grs, 20, 8192, "bf16", "bf16", "fp32")
    narrow.forward()
    loose = Case(grs, 20, 8201, "bf16", "bf16", "fp32")
    loose.forward()
    for call, status in ((lambda: quit_at(c, "bf16", "bf16", 10, 0, 0), inv), (lambda: quit_at(c, "bf16", "bf16", 3_000_000_000, 0, 0), inv),
                         (lambda: quit_at(c, "bf16", "bf16", 2_000_000, -1, 0), inv), (lambda: quit_at(c, "bf16", "bf16", 2_000_000, 0, -1), inv),
                         (lambda: quit_at(c, "bf16", "bf16", 2_000_000, 0, 0, dx=False), sh),
                         (lambda: quit_at(narrow, "bf16", "bf16", 2_000_000, 0, 0), sh), (lambda: quit_at(loose, "bf16", "bf16", 2_000_000, 0, 0), sh)):
        with pytest.raises(grs.GrsError) as e:
            call()
        assert e.value.status == status
