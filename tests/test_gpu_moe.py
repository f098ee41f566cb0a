"""Tokens sorted by expert and back, on the GPU, against numpy."""
import numpy as np
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


def stream():
    return torch.cuda.current_stream().cuda_stream


def sort(grs, s, ids):
    n = ids.numel()
    out = [torch.full((k,), -7, dtype=torch.int32, device="cuda") for k in (s.expert_end - s.expert_begin + 1, n, n)]
    ws = torch.full((grs.grs_moe_workspace_bytes(s) // 4 + 4,), -1, dtype=torch.int32, device="cuda")
    grs.grs_moe_sort(s, ids.data_ptr(), *(t.data_ptr() for t in out), ws.data_ptr(), stream())
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in out]


def sorted64(ids, begin, end):
    """(offsets, row_slot, slot_row) of a stable sort."""
    ids = ids.astype(np.int64)
    local = np.flatnonzero((ids >= begin) & (ids < end))
    order = local[np.argsort(ids[local], kind="stable")]
    row_slot = np.full(len(ids), -1)
    row_slot[:len(order)] = order
    slot_row = np.full(len(ids), -1)
    slot_row[order] = np.arange(len(order))
    counts = np.bincount(ids[local] - begin, minlength=end - begin)
    return np.concatenate([[0], np.cumsum(counts)]), row_slot, slot_row


@pytest.mark.parametrize("tokens,k", [(1, 1), (1, 8), (5, 4), (31, 1), (33, 3), (128, 1), (512, 8), (513, 8), (1000, 5), (4096, 1), (4097, 1),
                                      (20001, 6), (65536, 8)])
@pytest.mark.parametrize("experts,begin,end,kind", [(32, 0, 32, "any"), (32, 16, 32, "any"), (1, 0, 1, "any"), (1024, 0, 1024, "any"),
                                                    (257, 3, 200, "any"), (8, 0, 8, "one"), (8, 2, 4, "none"), (8, 0, 8, "wild"), (40, 0, 40, "runs")])
def test_sort(grs, tokens, k, experts, begin, end, kind):
    rng = np.random.default_rng(tokens * 31 + k + experts)
    n = tokens * k
    ids = rng.integers(0, experts, n)
    if kind == "one":
        ids[:] = 5
    elif kind == "none":
        ids[:] = 7
    elif kind == "wild":  # ids of no expert
        ids = rng.choice([-1, 0, 3, 7, 8, -2 ** 31, 2 ** 31 - 1], n)
    elif kind == "runs":
        ids = np.sort(ids)[::-1].copy()
    s = grs.make_moe(tokens, k, experts, begin, end, 8, 0)
    got = sort(grs, s, torch.from_numpy(ids.astype(np.int32)).cuda())
    for a, b in zip(got, sorted64(ids, begin, end)):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("experts,begin,end", [(1024, 0, 1024), (900, 100, 900), (3, 0, 3)])
def test_sort_of_many_slots(grs, experts, begin, end):
    """Tables of counts beyond what one block adds up by itself."""
    tokens, k = 250007, 8
    ids = np.random.default_rng(1).integers(0, experts, tokens * k).astype(np.int32)
    got = sort(grs, grs.make_moe(tokens, k, experts, begin, end, 8, 0), torch.from_numpy(ids).cuda())
    for a, b in zip(got, sorted64(ids, begin, end)):
        assert np.array_equal(a, b)


class Case:
    def __init__(self, grs, tokens, k, d, act, experts=6, begin=0, end=6, shift=0, seed=0):
        self.grs, self.tokens, self.k, self.d, self.act = grs, tokens, k, d, DT[act]
        self.s = grs.make_moe(tokens, k, experts, begin, end, d, 0 if act == "bf16" else 1)
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        ids = rng.integers(0, experts, tokens * k)
        self.rows = torch.from_numpy(sorted64(ids, begin, end)[2].astype(np.int32)).cuda()
        self.n = tokens * k
        self.shift = shift
        self.w = torch.rand(self.n, generator=self.g, device="cuda")
        self.w[self.rows < 0] = float("nan")  # not used

    def mat(self, rows, fill=None):
        buf = torch.full((rows * self.d + self.shift + 8,), float("nan"), dtype=self.act, device="cuda")
        m = buf[self.shift:self.shift + rows * self.d].view(rows, self.d)
        if fill is not None:
            m.copy_(torch.randn(rows, self.d, generator=self.g, device="cuda") * fill)
        return m

    def live(self):
        return self.rows[self.rows >= 0].long(), torch.nonzero(self.rows >= 0)[:, 0]


def close(got, want, bound):
    if got.dtype == torch.bfloat16:
        bound = bound + want.abs() * 2.0 ** -8 + 2.0 ** -126
    assert torch.isfinite(got).all()
    assert ((got.double() - want).abs() <= bound).all(), float(((got.double() - want).abs() - bound).max())


SHAPES = [(1, 1, 1), (1, 8, 2048), (3, 2, 7), (40, 3, 64), (17, 8, 515), (100, 1, 1032), (9, 5, 4100), (2, 20, 33), (300, 4, 2048), (5, 2, 9000), (1200, 6, 72)]


@pytest.mark.parametrize("tokens,k,d", SHAPES)
@pytest.mark.parametrize("act,begin,end,shift", [("bf16", 0, 6, 0), ("fp32", 0, 6, 0), ("bf16", 2, 5, 0), ("bf16", 0, 6, 1), ("fp32", 1, 2, 3)])
def test_vectors_there_and_back(grs, tokens, k, d, act, begin, end, shift):
    c = Case(grs, tokens, k, d, act, begin=begin, end=end, shift=shift, seed=tokens + d)
    rows, slots = c.live()
    rp, st = c.rows.data_ptr(), stream()
    x = c.mat(tokens, 1.0)
    xs = c.mat(c.n)
    grs.grs_moe_dispatch(c.s, x.data_ptr(), rp, xs.data_ptr(), st)
    want = torch.full_like(xs, float("nan"))
    want[rows] = x[slots // k]
    assert torch.equal(torch.nan_to_num(xs, nan=9.0), torch.nan_to_num(want, nan=9.0))  # rows without a slot are not written

    ys = c.mat(c.n, 0.5)
    on = (c.rows >= 0).view(tokens, k)
    w = torch.where(on, c.w.view(tokens, k), torch.zeros(())).double()
    take = lambda m: torch.where(on[:, :, None], m.double()[c.rows.clamp(min=0).long()].view(tokens, k, d), torch.zeros((), dtype=torch.float64))  # noqa: E731
    y = c.mat(tokens)
    grs.grs_moe_combine(c.s, ys.data_ptr(), rp, c.w.data_ptr(), y.data_ptr(), st)
    t = take(ys) * w[:, :, None]
    close(y, t.sum(1), (k + 1) * EPS32 * t.abs().sum(1))

    dx = c.mat(tokens)
    grs.grs_moe_dispatch_backward(c.s, ys.data_ptr(), rp, dx.data_ptr(), st)
    t = take(ys)
    close(dx, t.sum(1), k * EPS32 * t.abs().sum(1))

    dy = c.mat(tokens, 0.1)
    dys = c.mat(c.n)
    dw = torch.full((c.n,), float("nan"), device="cuda")
    grs.grs_moe_combine_backward(c.s, dy.data_ptr(), ys.data_ptr(), rp, c.w.data_ptr(), dys.data_ptr(), dw.data_ptr(), st)
    g = dy.double()[slots // k] * c.w[slots].double()[:, None]
    close(dys[rows], g, EPS32 * g.abs())
    dead = torch.ones(c.n, dtype=torch.bool, device="cuda")
    dead[rows] = False
    assert torch.isnan(dys[dead]).all()
    t = take(ys) * dy.double()[:, None, :]
    # products and sums in at most d / 32 + 32 roundings
    close(dw.view(tokens, k), t.sum(2), (d / 32 + 32) * EPS32 * t.abs().sum(2))
    assert (dw.view(tokens, k)[~on] == 0).all()
    dw2 = torch.empty_like(dw)
    grs.grs_moe_combine_backward(c.s, dy.data_ptr(), ys.data_ptr(), rp, c.w.data_ptr(), dys.data_ptr(), dw2.data_ptr(), st)
    assert torch.equal(dw, dw2)


@pytest.mark.parametrize("d", [64, 67])
def test_entries_outside_the_rows_stand_for_none(grs, d):
    c = Case(grs, 4, 2, d, "fp32", seed=1)
    c.rows = torch.tensor([0, 8, 2 ** 31 - 1, -1, -2 ** 31, 3, 5, 100], dtype=torch.int32, device="cuda")
    c.w = torch.rand(8, device="cuda")
    ys = c.mat(8, 1.0)
    y, dw, dys = c.mat(4), torch.empty(8, device="cuda"), c.mat(8)
    grs.grs_moe_combine(c.s, ys.data_ptr(), c.rows.data_ptr(), c.w.data_ptr(), y.data_ptr(), stream())
    assert torch.equal(y[0], ys[0] * c.w[0]) and (y[1] == 0).all() and torch.equal(y[2], ys[3] * c.w[5])
    grs.grs_moe_combine_backward(c.s, y.data_ptr(), ys.data_ptr(), c.rows.data_ptr(), c.w.data_ptr(), dys.data_ptr(), dw.data_ptr(), stream())
    assert (dw[[1, 2, 3, 4, 7]] == 0).all()
    assert torch.isnan(dys[[1, 2, 4, 6, 7]]).all() and torch.isfinite(dys[[0, 3, 5]]).all()


def test_gradients_against_differences(grs):
    """loss = sum(combine(f(dispatch(x)), w) * dy) with f(v) = v^2 / 2: against central differences in x and w."""
    tokens, k, d = 6, 3, 40
    c = Case(grs, tokens, k, d, "fp32", begin=0, end=6, seed=4)
    st, rp = stream(), c.rows.data_ptr()
    x, dy = c.mat(tokens, 1.0), c.mat(tokens, 1.0)
    xs, ys, y, dys, dx = c.mat(c.n), c.mat(c.n), c.mat(tokens), c.mat(c.n), c.mat(tokens)
    dw = torch.empty(c.n, device="cuda")

    def value():
        grs.grs_moe_dispatch(c.s, x.data_ptr(), rp, xs.data_ptr(), st)
        ys.copy_(xs * xs / 2)
        grs.grs_moe_combine(c.s, ys.data_ptr(), rp, c.w.data_ptr(), y.data_ptr(), st)
        return float((y.double() * dy.double()).sum())

    value()
    grs.grs_moe_combine_backward(c.s, dy.data_ptr(), ys.data_ptr(), rp, c.w.data_ptr(), dys.data_ptr(), dw.data_ptr(), st)
    dxs = dys * xs
    grs.grs_moe_dispatch_backward(c.s, dxs.data_ptr(), rp, dx.data_ptr(), st)
    for t, grad in ((x, dx), (c.w, dw)):
        keep, step = t.clone(), 1e-2
        v = torch.randn(t.shape, generator=c.g, device="cuda")
        want = float((grad.double() * v.double()).sum())
        t.copy_(keep + step * v)
        up = value()
        t.copy_(keep - step * v)
        down = value()
        t.copy_(keep)
        # the loss is quadratic: differences are exact but for fp32's rounding of about 100 terms of order 1
        assert abs((up - down) / (2 * step) - want) <= 1e3 * 16 * EPS32 / step


def test_rows_beyond_32_bits_of_elements(grs):
    """More than 2^31 elements of rows: the last tokens' rows, there and back."""
    tokens, k, d = 132000, 8, 2048
    s = grs.make_moe(tokens, k, 32, 0, 32, d, 0)
    rows = torch.arange(tokens * k, dtype=torch.int32, device="cuda").view(k, tokens).t().contiguous().view(-1)  # spread over all
    x = torch.zeros(tokens, d, dtype=torch.bfloat16, device="cuda")
    x[-50:] = torch.randn(50, d, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
    xs = torch.full((tokens * k, d), 3.0, dtype=torch.bfloat16, device="cuda")
    grs.grs_moe_dispatch(s, x.data_ptr(), rows.data_ptr(), xs.data_ptr(), stream())
    last = rows.view(tokens, k)[-50:].long()
    assert torch.equal(xs[last], x[-50:, None, :].expand(50, k, d))
    assert int((xs[rows.view(tokens, k)[:-50].reshape(-1)[::997].long()] != 0).sum()) == 0
    y = torch.empty_like(x)
    grs.grs_moe_dispatch_backward(s, xs.data_ptr(), rows.data_ptr(), y.data_ptr(), stream())
    assert torch.equal(y[-50:], (x[-50:].float() * k).to(torch.bfloat16))
    del xs, x, y
    torch.cuda.empty_cache()


def test_a_copy_keeps_every_bit(grs):
    """dispatch moves NaN payloads and signed zeros as they are, in both types and at any alignment."""
    for dt, code, word in ((torch.bfloat16, 0, torch.int16), (torch.float32, 1, torch.int32)):
        for d in (64, 67):
            g = torch.Generator(device="cuda").manual_seed(d)
            info = torch.iinfo(word)
            bits = torch.randint(info.min, info.max, (5, d), generator=g, device="cuda").to(word)
            s = grs.make_moe(5, 2, 4, 0, 4, d, code)
            rows = torch.randperm(10, generator=g, device="cuda").to(torch.int32)
            xs = torch.zeros(10, d, dtype=word, device="cuda")
            grs.grs_moe_dispatch(s, bits.data_ptr(), rows.data_ptr(), xs.data_ptr(), stream())
            assert torch.equal(xs[rows.long()], bits.repeat_interleave(2, 0))


def test_on_another_stream(grs):
    """Sort, dispatch and combine on a side stream only: what it waits for there is the result."""
    tokens, k, d = 3000, 4, 512
    g = torch.Generator(device="cuda").manual_seed(2)
    s = grs.make_moe(tokens, k, 16, 0, 16, d, 0)
    ids = torch.randint(0, 16, (tokens * k,), generator=g, device="cuda").to(torch.int32)
    x = torch.randn(tokens, d, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.full((tokens * k,), 0.25, device="cuda")
    off, rs, sr = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (17, tokens * k, tokens * k))
    ws = torch.zeros(grs.grs_moe_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    xs, y = torch.zeros(tokens * k, d, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    st = side.cuda_stream
    grs.grs_moe_sort(s, ids.data_ptr(), off.data_ptr(), rs.data_ptr(), sr.data_ptr(), ws.data_ptr(), st)
    grs.grs_moe_dispatch(s, x.data_ptr(), sr.data_ptr(), xs.data_ptr(), st)
    grs.grs_moe_combine(s, xs.data_ptr(), sr.data_ptr(), w.data_ptr(), y.data_ptr(), st)
    side.synchronize()
    assert torch.equal(y, x)  # four quarters of the token itself
    assert np.array_equal(sr.cpu().numpy(), sorted64(ids.cpu().numpy(), 0, 16)[2])


def test_no_tokens(grs):
    s = grs.make_moe(0, 2, 4, 0, 4, 16, 0)
    off = torch.full((5,), -1, dtype=torch.int32, device="cuda")
    grs.grs_moe_sort(s, None, off.data_ptr(), None, None, None, stream())
    assert (off.cpu() == 0).all()
    for call in (lambda: grs.grs_moe_dispatch(s, None, None, None, 0), lambda: grs.grs_moe_dispatch_backward(s, None, None, None, 0),
                 lambda: grs.grs_moe_combine(s, None, None, None, None, 0),
                 lambda: grs.grs_moe_combine_backward(s, None, None, None, None, None, None, 0)):
        call()


def test_refusals(grs):
    t = torch.zeros(4096, device="cuda")
    p = t.data_ptr()
    inv, sh, ali = grs.GRS_ERR_INVALID_ARG, grs.GRS_ERR_SHAPE, grs.GRS_ERR_ALIGNMENT
    raw = lambda tokens=4, k=2, b=0, e=4, d=16, dt=1: grs.grs_moe(tokens, k, b, e, d, dt, 0)  # noqa: E731
    disp = lambda s, x=p, r=p, y=p: grs.grs_moe_dispatch(s, x, r, y, 0)  # noqa: E731
    for call, status in ((lambda: disp(raw(tokens=-1)), sh), (lambda: disp(raw(k=0)), sh), (lambda: disp(raw(d=0)), sh), (lambda: disp(raw(d=(1 << 30) + 8)), sh),
                         (lambda: disp(raw(tokens=1 << 31)), sh), (lambda: disp(raw(tokens=1 << 30, k=2)), sh),
                         (lambda: disp(raw(b=-1)), inv), (lambda: disp(raw(b=4)), inv), (lambda: disp(raw(e=1025)), sh), (lambda: disp(raw(dt=2)), inv),
                         (lambda: disp(raw(), x=None), inv), (lambda: disp(raw(), r=None), inv), (lambda: disp(raw(), y=p + 2), ali),
                         (lambda: disp(raw(), r=p + 2), ali),
                         (lambda: grs.grs_moe_combine(raw(), p, p, None, p, 0), inv),
                         (lambda: grs.grs_moe_combine(raw(), p, p, p + 2, p, 0), ali),
                         (lambda: grs.grs_moe_combine_backward(raw(), p, p, p, p, p, None, 0), inv),
                         (lambda: grs.grs_moe_sort(raw(), p, None, p, p, p, 0), inv),
                         (lambda: grs.grs_moe_sort(raw(), p, p, p, p, p + 4, 0), ali),
                         (lambda: grs.make_moe(4, 2, 4, 0, 5, 16, 0), inv),
                         (lambda: grs.grs_moe_workspace_bytes(raw(k=-1)), inv)):
        with pytest.raises(grs.GrsError) as e:
            call()
        assert e.value.status == status
