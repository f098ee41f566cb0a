"""Row matrices of exactly a rank's rows: what its experts have, not
tokens * top_k, with guard words on both sides."""
import pytest
import torch

from test_gpu_moe import EPS32, Case, close, grs, stream  # noqa: F401

pytestmark = pytest.mark.gpu

GUARD = 5.0


def rows_of(c, rows, fill=None):
    """A matrix of `rows` vectors `shift` elements into a buffer of guards, and what lies around it."""
    n = rows * c.d
    buf = torch.full((c.shift + n + 1024,), GUARD, dtype=c.act, device="cuda")
    m = buf[c.shift:c.shift + n].view(rows, c.d)
    m.copy_(torch.randn(rows, c.d, generator=c.g, device="cuda") * fill) if fill is not None else m.fill_(float("nan"))
    return m, lambda: bool((buf[:c.shift] == GUARD).all() and (buf[c.shift + n:] == GUARD).all())


@pytest.mark.parametrize("tokens,k,d", [(1, 1, 7), (1, 3, 1), (40, 4, 67), (33, 6, 300), (17, 2, 515), (9, 5, 2051), (50, 3, 2052), (25, 8, 264)])
@pytest.mark.parametrize("act,shift", [("bf16", 0), ("bf16", 1), ("fp32", 0), ("fp32", 3)])
def test_a_rank_has_no_more_rows_than_its_experts(grs, tokens, k, d, act, shift):  # noqa: F811
    c = Case(grs, tokens, k, d, act, experts=8, begin=4, end=8, shift=shift, seed=tokens + d)
    rows, slots = c.live()
    n = max(1, len(rows))
    rp, st = c.rows.data_ptr(), stream()
    x = c.mat(tokens, 1.0)
    xs, around_xs = rows_of(c, n)
    grs.grs_moe_dispatch(c.s, x.data_ptr(), rp, xs.data_ptr(), st)
    assert torch.equal(xs[rows], x[slots // k]) and around_xs()

    on = (c.rows >= 0).view(tokens, k)
    w = torch.where(on, c.w.view(tokens, k), torch.zeros(())).double()
    ys, around_ys = rows_of(c, n, 0.5)
    took = torch.where(on[:, :, None], ys.double()[c.rows.clamp(min=0).long()].view(tokens, k, d), torch.zeros((), dtype=torch.float64))
    y, dx = c.mat(tokens), c.mat(tokens)
    grs.grs_moe_combine(c.s, ys.data_ptr(), rp, c.w.data_ptr(), y.data_ptr(), st)
    t = took * w[:, :, None]
    close(y, t.sum(1), (k + 1) * EPS32 * t.abs().sum(1))
    grs.grs_moe_dispatch_backward(c.s, ys.data_ptr(), rp, dx.data_ptr(), st)
    close(dx, took.sum(1), k * EPS32 * took.abs().sum(1))

    dy = c.mat(tokens, 0.1)
    dys, around_dys = rows_of(c, n)
    dw = torch.full((c.n,), float("nan"), device="cuda")
    grs.grs_moe_combine_backward(c.s, dy.data_ptr(), ys.data_ptr(), rp, c.w.data_ptr(), dys.data_ptr(), dw.data_ptr(), st)
    g = dy.double()[slots // k] * c.w[slots].double()[:, None]
    close(dys[rows], g, EPS32 * g.abs())
    t = took * dy.double()[:, None, :]
    close(dw.view(tokens, k), t.sum(2), (d / 32 + 32) * EPS32 * t.abs().sum(2))
    assert around_dys() and around_ys()
