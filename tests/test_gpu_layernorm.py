"""Layer norm forward and backward on the GPU against the formulas in 64 bits
and against differences of the forward pass."""
import pytest
import torch

pytestmark = pytest.mark.gpu

EPS32 = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def grs():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from gradient_reduction_sharded_gb300 import grs as g
    return g


def code(grs, name):
    return grs.GRS_DTYPE_BF16 if name == "bf16" else grs.GRS_DTYPE_FP32


def stream():
    return torch.cuda.current_stream().cuda_stream


def ptr(t):
    return None if t is None else t.data_ptr()


class Case:
    """Inputs in storage whose rows lie `pad` elements apart and start `shift` elements in, NaN around them."""

    def __init__(self, grs, rows, cols, act="fp32", par="fp32", grad="fp32", pad=0, shift=0, eps=1e-5, mean=0.3, std=1.5, seed=0):
        self.grs, self.rows, self.cols = grs, rows, cols
        self.act, self.par, self.grad = DT[act], DT[par], DT[grad]
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.ld = cols + pad
        self.shift = shift
        self.eps = eps
        self.x = self.rect(std, mean)
        self.dy = self.rect(1e-2, 0.0)
        self.w = (1 + 0.3 * torch.randn(cols, generator=self.gen, device="cuda")).to(self.par)
        self.b = (0.3 * torch.randn(cols, generator=self.gen, device="cuda")).to(self.par)
        self.shape = grs.make_norm(rows, cols, eps, code(grs, act), code(grs, par), code(grs, grad), self.ld, self.ld, self.ld, self.ld)
        self.ws = torch.full((grs.grs_layernorm_workspace_bytes(self.shape) // 4 + 4,), float("nan"), device="cuda")
        self.mean = torch.full((rows,), float("nan"), device="cuda")
        self.rstd = torch.full((rows,), float("nan"), device="cuda")

    def blank(self):
        return torch.full((self.rows * self.ld + self.shift + 8,), float("nan"), dtype=self.act, device="cuda")

    def view(self, buf):
        return buf[self.shift:self.shift + self.rows * self.ld].view(self.rows, self.ld)[:, :self.cols]

    def rect(self, std, mean):
        v = self.view(self.blank())
        v.copy_(torch.randn(self.rows, self.cols, generator=self.gen, device="cuda") * std + mean)
        return v

    def forward(self, w=True, b=True):
        buf = self.blank()
        y = self.view(buf)
        self.grs.grs_layernorm_forward(self.shape, self.x.data_ptr(), ptr(self.w if w else None), ptr(self.b if b else None), y.data_ptr(),
                                       self.mean.data_ptr(), self.rstd.data_ptr(), stream())
        torch.cuda.synchronize()
        self.untouched(buf)
        return y

    def untouched(self, buf):
        """Nothing is written between or around the rows."""
        mask = torch.ones(buf.shape, dtype=torch.bool, device="cuda")
        mask[self.shift:self.shift + self.rows * self.ld].view(self.rows, self.ld)[:, :self.cols] = False
        assert torch.isnan(buf[mask]).all()

    def backward(self, w=True, dx=True, dw=True, db=True):
        buf = self.blank()
        gx = self.view(buf)
        gw = torch.full((self.cols,), float("nan"), dtype=self.grad, device="cuda")
        gb = gw.clone()
        self.grs.grs_layernorm_backward(self.shape, self.dy.data_ptr(), self.x.data_ptr(), ptr(self.w if w else None), self.mean.data_ptr(),
                                        self.rstd.data_ptr(), gx.data_ptr() if dx else None, gw.data_ptr() if dw else None,
                                        gb.data_ptr() if db else None, self.ws.data_ptr(), stream())
        torch.cuda.synchronize()
        self.untouched(buf)
        return gx, gw, gb


def check(got, want, bound, what):
    """Within `bound` of the 64-bit value, plus the rounding to bf16 where that is the type."""
    if got.dtype == torch.bfloat16:
        bound = bound + want.abs() * 2.0 ** -8 + 2.0 ** -126
    off = (got.double() - want).abs()
    assert torch.isfinite(got).all(), what
    assert (off <= bound).all(), (what, float((off - bound).max()))


SHAPES = [(1, 1), (1, 16), (1, 2048), (3, 7), (64, 32), (5, 128), (33, 1024), (17, 1027), (29, 1000), (4, 4096), (2, 9001), (3, 16384),
          (2, 40000), (70001, 24), (3000, 130), (700, 2048)]


def forward64(c, w=True, b=True):
    x = c.x.double()
    mean = x.mean(1, keepdim=True)
    var = (x - mean).square().mean(1, keepdim=True)
    rstd = 1 / (var + c.eps).sqrt()
    h = (x - mean) * rstd
    return h * (c.w.double() if w else 1.0) + (c.b.double() if b else 0.0), mean[:, 0], rstd[:, 0], h


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("act,par,grad,pad,shift", [("fp32", "fp32", "fp32", 0, 0), ("bf16", "bf16", "bf16", 0, 0), ("bf16", "fp32", "fp32", 8, 0),
                                                    ("bf16", "bf16", "fp32", 3, 1), ("fp32", "bf16", "bf16", 5, 3)])
def test_against_64_bits(grs, rows, cols, act, par, grad, pad, shift):
    c = Case(grs, rows, cols, act, par, grad, pad, shift, seed=rows * 7 + cols)
    # fp32 sums of C terms in partial sums of at most C / 32 each; a row's own conditioning is (1 + max |x| rstd)
    k = (64 + cols / 32) * EPS32
    y, mean, rstd, h = forward64(c)
    got = c.forward()
    big = c.x.double().abs().amax(1, keepdim=True)
    cond = 1 + big * rstd[:, None]
    check(got, y, k * cond * (1 + h.abs()) * c.w.double().abs().amax() + k * c.b.double().abs(), "y")
    check(c.mean, mean, k * big[:, 0], "mean")
    check(c.rstd, rstd, k * cond[:, 0] * rstd, "rstd")
    gx, gw, gb = c.backward()
    # the backward pass takes the kept statistics as they are
    mean, rstd = c.mean.double()[:, None], c.rstd.double()[:, None]
    h = (c.x.double() - mean) * rstd
    dy = c.dy.double()
    dh = dy * c.w.double()
    dx = rstd * (dh - dh.mean(1, keepdim=True) - h * (dh * h).mean(1, keepdim=True))
    check(gx, dx, k * cond * rstd * dh.abs().amax(1, keepdim=True) * (1 + h.abs()) ** 2, "dx")
    k = (128 + rows / 64) * EPS32  # rows in partial sums, then the partial sums
    check(gw, (dy * h).sum(0), k * (dy.abs() * (h.abs() + cond)).sum(0), "dw")
    check(gb, dy.sum(0), k * dy.abs().sum(0), "db")
    again = c.backward()
    for a, b in zip((gx, gw, gb), again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("cols", [24, 1024, 1027])
@pytest.mark.parametrize("act", ["fp32", "bf16"])
def test_optional_arguments(grs, cols, act):
    c = Case(grs, 37, cols, act, seed=3)
    y, mean, rstd, h = forward64(c, w=False, b=False)
    k = (64 + cols / 32) * EPS32
    cond = 1 + c.x.double().abs().amax(1, keepdim=True) * rstd[:, None]
    check(c.forward(w=False, b=False), y, k * cond * (1 + h.abs()), "y")
    full = c.backward(w=False)
    for only in (dict(dx=True, dw=False, db=False), dict(dx=False, dw=True, db=False), dict(dx=False, dw=False, db=True),
                 dict(dx=False, dw=True, db=True), dict(dx=True, dw=True, db=False)):
        got = c.backward(w=False, **only)
        for name, a, b in zip(("dx", "dw", "db"), got, full):
            if only[name]:
                assert torch.equal(a, b), (only, name)
            else:
                assert torch.isnan(a).all()
    # statistics not kept
    y1 = torch.empty(37, cols, dtype=c.act, device="cuda")
    grs.grs_layernorm_forward(c.shape, c.x.data_ptr(), None, None, y1.data_ptr(), None, None, stream())
    assert torch.equal(y1, c.forward(w=False, b=False))


def test_no_rows_gives_zero_parameter_gradients(grs):
    c = Case(grs, 0, 100)
    _, gw, gb = c.backward()
    assert (gw == 0).all() and (gb == 0).all()
    grs.grs_layernorm_forward(c.shape, None, None, None, None, None, None, stream())


@pytest.mark.parametrize("cols", [64, 1003, 4096])
def test_gradients_against_differences(grs, cols):
    """Central differences of sum(y * dy) along random directions of x, w and b."""
    c = Case(grs, 3, cols, "fp32", seed=5)
    c.dy.mul_(100)
    c.forward()
    gx, gw, gb = c.backward()
    value = lambda: float((c.forward().double() * c.dy.double()).sum())  # noqa: E731
    for t, g in ((c.x, gx), (c.w, gw), (c.b, gb)):
        keep = t.clone()
        v = torch.randn(t.shape, generator=c.gen, device="cuda")
        step = 1e-2
        t.copy_(keep + step * v)
        up = value()
        t.copy_(keep - step * v)
        down = value()
        t.copy_(keep)
        want = float((g.double() * v.double()).sum())
        # third-order term of the difference (step^2), and the forward pass's rounding over 2 step
        size = float(c.dy.double().norm()) * float(v.double().norm())
        assert abs((up - down) / (2 * step) - want) <= size * (step ** 2 + 64 * EPS32 / step)


def test_large_mean_and_constant_rows(grs):
    c = Case(grs, 8, 512, "fp32", mean=1000.0, std=1.0, seed=7)
    c.x[3] = 5.0
    y, mean, rstd, h = forward64(c)
    got = c.forward()
    cond = 1 + c.x.double().abs().amax(1, keepdim=True) * rstd[:, None]
    check(got, y, (64 + 16) * EPS32 * cond * (1 + h.abs()) * c.w.double().abs().amax() + EPS32 * 64, "y")
    assert (got[3] == c.b).all()  # h is exactly 0
    assert torch.isfinite(c.backward()[0]).all()


@pytest.mark.parametrize("cols", [128, 2048, 1001])
def test_nan_and_infinity_stay_in_their_row(grs, cols):
    c = Case(grs, 6, cols, "bf16", "bf16", seed=8)
    clean = c.forward().clone()
    c.x[2, 5] = float("nan")
    c.x[4, 0] = float("inf")
    got = c.forward()
    for r in range(6):
        if r in (2, 4):
            assert torch.isnan(got[r]).any()
        else:
            assert torch.equal(got[r], clean[r])


def test_on_another_stream_and_in_a_graph(grs):
    """Both passes on a side stream, and replayed from a captured graph on new inputs: the same bits as on the default stream."""
    c = Case(grs, 700, 2048, "bf16", "bf16", "bf16", seed=9)
    want = [c.forward().clone(), *(t.clone() for t in c.backward())]
    y, gx = torch.empty_like(c.x), torch.empty_like(c.x)
    gw, gb = torch.empty_like(c.w), torch.empty_like(c.w)

    def both(st):
        grs.grs_layernorm_forward(c.shape, c.x.data_ptr(), c.w.data_ptr(), c.b.data_ptr(), y.data_ptr(), c.mean.data_ptr(), c.rstd.data_ptr(), st)
        grs.grs_layernorm_backward(c.shape, c.dy.data_ptr(), c.x.data_ptr(), c.w.data_ptr(), c.mean.data_ptr(), c.rstd.data_ptr(), gx.data_ptr(),
                                   gw.data_ptr(), gb.data_ptr(), c.ws.data_ptr(), st)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both(side.cuda_stream)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((y, gx, gw, gb), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(stream())
    c.x.copy_(c.x.flip(0))
    c.dy.copy_(c.dy.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want[0].flip(0)) and torch.equal(gx, want[1].flip(0))


def test_rows_beyond_32_bits_of_elements(grs):
    """An offset past 2^31 elements: the last rows of a strided view."""
    rows, cols, ld = 5, 64, 1 << 29
    buf = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    x = buf.view(rows, ld)[:, :cols]
    x.copy_(torch.randn(rows, cols, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)))
    y = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    s = grs.make_norm(rows, cols, 1e-5, 0, 0, 0, ld_x=ld)
    grs.grs_layernorm_forward(s, x.data_ptr(), None, None, y.data_ptr(), None, None, stream())
    x64 = x.double()
    want = (x64 - x64.mean(1, keepdim=True)) / (x64.var(1, correction=0, keepdim=True) + 1e-5).sqrt()
    check(y, want, 1e-5, "y")


def test_refusals(grs):
    c = Case(grs, 4, 32)
    p = c.x.data_ptr()
    inv, sh, ali = grs.GRS_ERR_INVALID_ARG, grs.GRS_ERR_SHAPE, grs.GRS_ERR_ALIGNMENT
    mk = lambda rows=4, cols=32, eps=1e-5, dt=1, pd=1, gd=1, **ld: grs.make_norm(rows, cols, eps, dt, pd, gd, **ld)  # noqa: E731
    fwd = lambda s, x=p, w=p, y=p: grs.grs_layernorm_forward(s, x, w, None, y, None, None, 0)  # noqa: E731
    bwd = lambda s, dy=p, mean=p, dw=p, ws=p, dx=p: grs.grs_layernorm_backward(s, dy, p, p, mean, p, dx, dw, None, ws, 0)  # noqa: E731
    for call, status in ((lambda: fwd(mk(rows=-1)), sh), (lambda: fwd(mk(cols=0)), sh), (lambda: fwd(mk(cols=(1 << 30) + 1)), sh), (lambda: fwd(mk(ld_x=31)), sh), (lambda: fwd(mk(ld_dx=-1)), sh),
                         (lambda: fwd(mk(eps=-1.0)), inv), (lambda: fwd(mk(eps=float("nan"))), inv), (lambda: fwd(mk(dt=2)), inv),
                         (lambda: fwd(mk(pd=-1)), inv), (lambda: fwd(mk(gd=9)), inv), (lambda: fwd(mk(), x=None), inv),
                         (lambda: fwd(mk(), y=None), inv), (lambda: fwd(mk(), x=p + 2), ali), (lambda: fwd(mk(), w=p + 1), ali),
                         (lambda: bwd(mk(), dy=None), inv), (lambda: bwd(mk(), mean=None), inv), (lambda: bwd(mk(), ws=None), inv),
                         (lambda: bwd(mk(), ws=p + 4), ali), (lambda: bwd(mk(), dw=p + 2), ali), (lambda: bwd(mk(), dx=p + 1), ali),
                         (lambda: grs.grs_layernorm_workspace_bytes(mk(cols=0)), inv)):
        with pytest.raises(grs.GrsError) as e:
            call()
        assert e.value.status == status
