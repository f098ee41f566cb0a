"""Layer norm and the expert calls on matrices of more than 2^31 elements:
what lies at their ends, each path once."""
import pytest
import torch

from test_gpu_layernorm import DT, EPS32, check, code, forward64, grs  # noqa: F401
from test_gpu_layernorm_wide import gradients64
from test_gpu_moe import close

pytestmark = pytest.mark.gpu

TAIL = 40


def st():
    return torch.cuda.current_stream().cuda_stream


class Tail:
    """The last rows of a matrix whose other rows are zeros."""

    def __init__(self, cols, act, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.rows, self.cols, self.eps = TAIL, cols, 1e-5
        self.x = (torch.randn(TAIL, cols, generator=g, device="cuda") * 1.5 + 0.3).to(DT[act])
        self.dy = (torch.randn(TAIL, cols, generator=g, device="cuda") * 1e-2).to(DT[act])
        self.w = (1 + 0.3 * torch.randn(cols, generator=g, device="cuda")).to(DT[act])
        self.b = (0.3 * torch.randn(cols, generator=g, device="cuda")).to(DT[act])


# blocks and clusters of whole rows, loose rows in registers and a block a row
@pytest.mark.parametrize("cols,act", [(2048, "bf16"), (128, "bf16"), (8200, "bf16"), (20000, "bf16"), (4104, "fp32"), (2051, "bf16"), (9001, "bf16"), (16387, "fp32")])
def test_layer_norm(grs, cols, act):  # noqa: F811
    rows = (1 << 31) // cols + 3 * TAIL
    size = rows * cols * DT[act].itemsize
    if torch.cuda.mem_get_info()[0] < 5 * size:
        pytest.skip("needs up to 44 GB of device memory")
    c = Tail(cols, act, cols)
    x, dy, out = (torch.zeros(rows, cols, dtype=DT[act], device="cuda") for _ in range(3))
    x[-TAIL:], dy[-TAIL:] = c.x, c.dy
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    s = grs.make_norm(rows, cols, c.eps, code(grs, act), code(grs, act), grs.GRS_DTYPE_FP32)
    ws = torch.empty(grs.grs_layernorm_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    grs.grs_layernorm_forward(s, x.data_ptr(), c.w.data_ptr(), c.b.data_ptr(), out.data_ptr(), mean.data_ptr(), rstd.data_ptr(), st())
    want, m64, r64, h = forward64(c)
    k = (64 + cols / 32) * EPS32
    big = c.x.double().abs().amax(1, keepdim=True)
    cond = 1 + big * r64[:, None]
    check(out[-TAIL:], want, k * cond * (1 + h.abs()) * c.w.double().abs().amax() + k * c.b.double().abs(), "y")
    check(mean[-TAIL:], m64, k * big[:, 0], "mean")
    check(rstd[-TAIL:], r64, k * cond[:, 0] * r64, "rstd")
    assert torch.equal(out[rows // 2], c.b) and torch.equal(out[-TAIL - 1], c.b)  # rows of zeros
    c.mean, c.rstd = mean[-TAIL:], rstd[-TAIL:]
    out.fill_(7.0)
    dw, db = torch.zeros(cols, device="cuda"), torch.zeros(cols, device="cuda")
    grs.grs_layernorm_backward(s, dy.data_ptr(), x.data_ptr(), c.w.data_ptr(), mean.data_ptr(), rstd.data_ptr(), out.data_ptr(), dw.data_ptr(),
                               db.data_ptr(), ws.data_ptr(), st())
    for got, (want, bound), what in zip((out[-TAIL:], dw, db), gradients64(c), ("dx", "dw", "db")):
        check(got, want, bound, what)
    assert not out[:-TAIL].any()
    assert grs.grs_layernorm_check_device_errors(st()) == grs.GRS_OK
    del x, dy, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("d,act,code_", [(2048, "bf16", 0), (2051, "bf16", 0), (2052, "fp32", 1)])
def test_experts_there_and_back(grs, d, act, code_):  # noqa: F811
    tokens, k = 132000, 8
    size = tokens * k * d * DT[act].itemsize
    if torch.cuda.mem_get_info()[0] < 4 * size:
        pytest.skip("needs up to 36 GB of device memory")
    g = torch.Generator(device="cuda").manual_seed(d)
    s = grs.make_moe(tokens, k, 32, 0, 32, d, code_)
    rows = torch.arange(tokens * k, dtype=torch.int32, device="cuda").view(k, tokens).t().contiguous()  # a token's rows spread over all
    last = rows[-TAIL:].long()
    w = torch.rand(tokens, k, generator=g, device="cuda")
    x = torch.zeros(tokens, d, dtype=DT[act], device="cuda")
    x[-TAIL:] = torch.randn(TAIL, d, generator=g, device="cuda").to(DT[act])
    ys = torch.zeros(tokens * k, d, dtype=DT[act], device="cuda")
    ys[last.view(-1)] = torch.randn(TAIL * k, d, generator=g, device="cuda").to(DT[act])
    xs, y = torch.full_like(ys, 3.0), torch.full_like(x, 3.0)
    grs.grs_moe_dispatch(s, x.data_ptr(), rows.data_ptr(), xs.data_ptr(), st())
    assert torch.equal(xs[last], x[-TAIL:, None, :].expand(TAIL, k, d))
    assert not xs[rows[:-TAIL].reshape(-1)[::997].long()].any()
    took = ys[last].double()
    wt = w[-TAIL:].double()[:, :, None]
    grs.grs_moe_combine(s, ys.data_ptr(), rows.data_ptr(), w.data_ptr(), y.data_ptr(), st())
    close(y[-TAIL:], (took * wt).sum(1), (k + 1) * EPS32 * (took * wt).abs().sum(1))
    assert not y[:-TAIL].any()
    grs.grs_moe_dispatch_backward(s, ys.data_ptr(), rows.data_ptr(), y.data_ptr(), st())
    close(y[-TAIL:], took.sum(1), k * EPS32 * took.abs().sum(1))
    dys, dw = xs.fill_(3.0), torch.full((tokens, k), 3.0, device="cuda")
    grs.grs_moe_combine_backward(s, x.data_ptr(), ys.data_ptr(), rows.data_ptr(), w.data_ptr(), dys.data_ptr(), dw.data_ptr(), st())
    want = x[-TAIL:].double()[:, None, :] * wt
    close(dys[last], want, EPS32 * want.abs())
    t = took * x[-TAIL:].double()[:, None, :]
    close(dw[-TAIL:], t.sum(2), (d / 32 + 32) * EPS32 * t.abs().sum(2))
    assert not dw[:-TAIL].any() and not dys[rows[:-TAIL].reshape(-1)[::997].long()].any()
    del x, ys, xs, y, dys
    torch.cuda.empty_cache()
