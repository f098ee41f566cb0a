"""Layer norm where the launch changes shape: rows wider than the registers of
a block (shared by the blocks of a cluster), and matrices beyond L2, down to
the narrowest rows.  Bounds as in the tests of ordinary sizes."""
import pytest
import torch

from test_gpu_layernorm import EPS32, Case, check, forward64, grs  # noqa: F401

pytestmark = pytest.mark.gpu

TYPES = [("fp32", "fp32", "fp32", 0, 0), ("bf16", "bf16", "bf16", 0, 0), ("bf16", "fp32", "fp32", 8, 0), ("bf16", "bf16", "fp32", 3, 1),
         ("fp32", "bf16", "bf16", 5, 3)]


def gradients64(c, w=True):
    mean, rstd = c.mean.double()[:, None], c.rstd.double()[:, None]
    h = (c.x.double() - mean) * rstd
    dy = c.dy.double()
    dh = dy * (c.w.double() if w else 1.0)
    dx = rstd * (dh - dh.mean(1, keepdim=True) - h * (dh * h).mean(1, keepdim=True))
    cond = 1 + c.x.double().abs().amax(1, keepdim=True) * rstd
    k = (64 + c.cols / 32) * EPS32
    dx_bound = k * cond * rstd * dh.abs().amax(1, keepdim=True) * (1 + h.abs()) ** 2
    k = (128 + c.rows / 64) * EPS32
    return (dx, dx_bound), ((dy * h).sum(0), k * (dy.abs() * (h.abs() + cond)).sum(0)), (dy.sum(0), k * dy.abs().sum(0))


# one row, fewer rows than clusters, several a cluster; shares that end in a part of a chunk; past what a cluster holds
@pytest.mark.parametrize("rows,cols", [(1, 8200), (1, 32768), (3, 8193), (40, 12007), (301, 16384), (130, 20008), (64, 32769), (5, 65536), (4, 65537)])
@pytest.mark.parametrize("act,par,grad,pad,shift", TYPES)
def test_wide_rows(grs, rows, cols, act, par, grad, pad, shift):  # noqa: F811
    c = Case(grs, rows, cols, act, par, grad, pad, shift, seed=rows + cols)
    c.forward()
    got = c.backward()
    for g, (want, bound), what in zip(got, gradients64(c), ("dx", "dw", "db")):
        check(g, want, bound, what)
    for a, b in zip(got, c.backward()):
        assert torch.equal(a, b)


# fp32 rows that one block could hold, shared where they are many
@pytest.mark.parametrize("rows,cols", [(607, 4104), (608, 4104), (1500, 8192), (700, 5128), (610, 4097)])
def test_fp32_rows_of_a_cluster_or_a_block(grs, rows, cols):  # noqa: F811
    test_wide_rows(grs, rows, cols, "fp32", "fp32", "fp32", 0, 0)


@pytest.mark.parametrize("cols", [8200, 16387])
@pytest.mark.parametrize("act", ["fp32", "bf16"])
def test_wide_rows_optional_arguments(grs, cols, act):  # noqa: F811
    c = Case(grs, 23, cols, act, act, "fp32", seed=cols)
    c.forward(w=False, b=False)
    full = c.backward(w=False)
    for g, (want, bound), what in zip(full, gradients64(c, w=False), ("dx", "dw", "db")):
        check(g, want, bound, what)
    for dx, dw, db in ((True, False, False), (False, True, False), (False, False, True), (False, True, True), (True, False, True)):
        part = c.backward(w=False, dx=dx, dw=dw, db=db)
        for want, got, asked in zip(full, part, (dx, dw, db)):
            if asked:
                check(got, want.double(), 64 * EPS32 * want.double().abs().amax(), "part")
            else:
                assert torch.isnan(got).all()


def test_wide_rows_nan_and_infinity_stay_in_their_row(grs):  # noqa: F811
    c = Case(grs, 9, 16384, "bf16", "bf16", "fp32")
    c.x[2, 5] = float("nan")
    c.x[6, 16383] = float("inf")
    c.forward()
    gx = c.backward()[0]
    bad = torch.isnan(gx).any(1)
    assert bad.tolist() == [i in (2, 6) for i in range(9)]


# widths that no other test has: the first call of their launch shape is the captured one
@pytest.mark.parametrize("act,cols", [("bf16", 10000), ("fp32", 10400)])
def test_wide_rows_in_a_graph_on_another_stream(grs, act, cols):  # noqa: F811
    c = Case(grs, 150, cols, act, act, "fp32", seed=3)
    c.forward()
    gx, gw, gb = torch.full_like(c.x, float("nan")), torch.zeros(cols, device="cuda"), torch.zeros(cols, device="cuda")
    shape = grs.make_norm(150, cols, c.eps, *[grs.GRS_DTYPE_BF16 if act == "bf16" else grs.GRS_DTYPE_FP32] * 2, grs.GRS_DTYPE_FP32)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        grs.grs_layernorm_backward(shape, c.dy.data_ptr(), c.x.data_ptr(), c.w.data_ptr(), c.mean.data_ptr(), c.rstd.data_ptr(), gx.data_ptr(),
                                   gw.data_ptr(), gb.data_ptr(), c.ws.data_ptr(), torch.cuda.current_stream().cuda_stream)
    for _ in range(3):
        gx.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for g, (want, bound), what in zip((gx, gw, gb), gradients64(c), ("dx", "dw", "db")):
            check(g, want, bound, what)


# more than 64 MB of x: the forward pass takes other blocks
@pytest.mark.parametrize("cols", [1, 7, 16, 33, 768, 2560, 5120])
@pytest.mark.parametrize("act,pad,shift", [("fp32", 0, 0), ("bf16", 0, 0), ("bf16", 1, 1), ("fp32", 3, 1)])
def test_forward_beyond_l2(grs, cols, act, pad, shift):  # noqa: F811
    size = 4 if act == "fp32" else 2
    rows = (68 << 20) // (cols * size)
    c = Case(grs, rows, cols, act, "fp32", "fp32", pad, shift, seed=cols)
    y = c.forward()
    k = (64 + cols / 32) * EPS32
    take = torch.cat([torch.arange(0, min(rows, 3000), device="cuda"), torch.randint(0, rows, (3000,), device="cuda"),
                      torch.arange(max(0, rows - 3000), rows, device="cuda")])
    part = Case.__new__(Case)
    part.__dict__.update(c.__dict__)
    part.x = c.x[take]
    want, mean, rstd, h = forward64(part)
    big = part.x.double().abs().amax(1, keepdim=True)
    cond = 1 + big * rstd[:, None]
    check(y[take], want, k * cond * (1 + h.abs()) * c.w.double().abs().amax() + k * c.b.double().abs(), "y")
    check(c.mean[take], mean, k * big[:, 0], "mean")
    check(c.rstd[take], rstd, k * cond[:, 0] * rstd, "rstd")
    assert torch.isfinite(y).all()
    assert torch.equal(y, c.forward())
