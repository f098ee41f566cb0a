"""Norms of queries and keys with the rotation against 64 bits: dimensions,
parts of a head turned, both kinds of pairs, far positions, heads inside wider
rows, in place."""
import itertools

import pytest
import torch

from operators_support import DT, binding, close, dtype_code, half, ptr, stream

pytestmark = pytest.mark.gpu

EPS = 1e-6
# Roundings that an element meets, in fp32's half steps: the sum of squares in chains of at most 32 + 8 additions
# (a lane has at most 1024 / 32 elements), its root and reciprocal, four products, sine and cosine (2 units each) of an
# angle to 2^-23, two products and their sum; the last three relative to both elements of a pair.
UNITS = 64 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


class Case:
    def __init__(self, t, hq, hk, d, rot, act="bf16", par="bf16", grad="bf16", pairs=False, far=0, pad=None, weights=True, seed=0, base=1e4, shift=0):
        grs = binding()
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.t, self.h, self.d, self.rot, self.act, self.grad, self.pairs = t, (hq, hk), d, rot, act, grad, pairs

        def rows(width, extra, std):
            wide = torch.full((t * (width + extra) + shift + 8,), 7.0, dtype=DT[act], device="cuda")
            m = wide[shift:shift + t * (width + extra)].view(t, width + extra)
            m[:, :width] = torch.randn(t, width, generator=g, device="cuda") * std
            return m

        extra = 0 if pad is None else pad
        self.ld = [hq * d + extra, hk * d + extra, hq * d, hk * d]
        self.x = [rows(h * d, extra, 2.0) for h in self.h]
        self.dy = [rows(h * d, 0, 0.3) for h in self.h]
        self.w = [(1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(DT[par]) if weights else None for _ in range(2)]
        self.pos = (torch.randint(-50, 5000, (t,), generator=g, device="cuda") + far).to(torch.int32)
        self.inv = [base ** (-2 * i / max(1, rot)) for i in range(rot // 2)]
        self.turns = torch.tensor(grs.grs_rope_turns(self.inv), dtype=torch.uint64, device="cuda")
        self.shape = grs.make_qk_norm(t, hq, hk, d, rot, EPS, dtype_code(act), dtype_code(par), dtype_code(grad), pairs, *self.ld)
        self.ws = torch.full((max(16, grs.grs_qk_norm_workspace_bytes(self.shape)),), 0xFF, dtype=torch.uint8, device="cuda")

    def tail(self):
        return (ptr(self.w[0]), ptr(self.w[1]), ptr(self.pos), ptr(self.turns))

    def forward(self, out=None):
        o = out or [torch.full((self.t, h * self.d), 7.0, dtype=DT[self.act], device="cuda") for h in self.h]
        binding().grs_qk_norm_forward(self.shape, ptr(self.x[0]), ptr(self.x[1]), *self.tail(), ptr(o[0]), ptr(o[1]), stream())
        return o

    def backward(self, dx=True, dw=True):
        dxs = [torch.full_like(x, 7.0) if dx else None for x in self.x]
        dws = [torch.full((self.d,), 7.0, dtype=DT[self.grad], device="cuda") if dw else None for _ in range(2)]
        binding().grs_qk_norm_backward(self.shape, ptr(self.dy[0]), ptr(self.dy[1]), ptr(self.x[0]), ptr(self.x[1]), *self.tail(),
                                       ptr(dxs[0]), ptr(dxs[1]), ptr(dws[0]), ptr(dws[1]), ptr(self.ws), stream())
        return dxs, dws

    # 64 bits -------------------------------------------------------------
    def heads(self, m, i):
        return m[:, :self.h[i] * self.d].double().reshape(self.t, self.h[i], self.d)

    def pair(self, u):
        z = u[..., :self.rot]
        return (z[..., 0::2], z[..., 1::2]) if self.pairs else z.chunk(2, -1) if self.rot else (z, z)

    def join(self, a, b, rest):
        z = torch.stack((a, b), -1).flatten(-2) if self.pairs else torch.cat((a, b), -1)
        return torch.cat((z, rest[..., self.rot:]), -1)

    def turned(self, u, back=False, size=False):
        """u turned; size: the magnitudes that meet in each element."""
        angle = self.pos.double()[:, None, None] * torch.tensor(self.inv, dtype=torch.float64, device="cuda")
        c, s = angle.cos(), angle.sin() * (-1 if back else 1)
        a, b = self.pair(u)
        if size:
            return self.join(a.abs() + b.abs(), a.abs() + b.abs(), u.abs())
        return self.join(a * c - b * s, a * s + b * c, u)

    def check(self):
        o = self.forward()
        dxs, dws = self.backward()
        assert binding().grs_operators_check_device_errors(stream()) == binding().GRS_OK
        for i in range(2):
            if not self.h[i]:
                assert bool((dws[i] == 0).all())
                continue
            x, dy = self.heads(self.x[i], i), self.heads(self.dy[i], i)
            w = self.w[i].double() if self.w[i] is not None else torch.ones(self.d, dtype=torch.float64, device="cuda")
            r = 1 / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
            h = x * r
            want = self.turned(h * w)
            close(o[i].view(x.shape), want, self.turned(h * w, size=True) * UNITS + want.abs() * half(self.act), ("out", i))
            du, size = self.turned(dy, back=True), self.turned(dy, back=True, size=True)
            dh, m = du * w, (du * w * h).mean(-1, keepdim=True)
            want = r * (dh - h * m)
            most = r * (size * w.abs() + h.abs() * (size * w.abs() * h.abs()).mean(-1, keepdim=True))
            width = self.h[i] * self.d
            close(dxs[i][:, :width].reshape(x.shape), want, most * UNITS + want.abs() * half(self.act), ("dx", i))
            assert bool((dxs[i][:, width:] == 7).all())
            want, most = (du * h).sum((0, 1)), (size * h.abs()).sum((0, 1))
            # a chain has at most as many additions as there are heads, and 64 roundings before it
            close(dws[i], want, most * (self.t * self.h[i] * 2.0 ** -24 + UNITS) + want.abs() * half(self.grad), ("dw", i))


@pytest.mark.parametrize("act, par, grad", [("bf16", "bf16", "bf16"), ("bf16", "fp32", "fp32"), ("bf16", "bf16", "fp32"), ("fp32", "fp32", "fp32"),
                                            ("fp32", "bf16", "bf16")])
@pytest.mark.parametrize("d, rot", [(128, 128), (128, 64), (64, 64), (256, 256), (96, 96), (80, 40), (32, 32), (1, 0), (5, 4), (130, 130), (1024, 1024), (192, 0)])
def test_dimensions_and_types(d, rot, act, par, grad):
    for pairs in (False, True):
        Case(37, 4, 2, d, rot, act, par, grad, pairs).check()


@pytest.mark.parametrize("t, hq, hk", [(1, 1, 1), (1, 16, 16), (3, 32, 4), (2, 0, 3), (2, 5, 0), (1000, 7, 1), (5000, 2, 1)])
@pytest.mark.parametrize("d", [64, 128, 80])
def test_tokens_and_heads(t, hq, hk, d):
    Case(t, hq, hk, d, d, "bf16", "bf16", "fp32").check()
    Case(t, hq, hk, d, d // 2, "fp32", "fp32", "fp32", pairs=True).check()


@pytest.mark.parametrize("pad, shift", [(8, 0), (64, 0), (3, 0), (0, 1), (8, 4)])
@pytest.mark.parametrize("act", ["bf16", "fp32"])
def test_heads_inside_wider_rows_and_any_alignment(pad, shift, act):
    Case(50, 3, 2, 64, 64, act, "fp32", "fp32", pad=pad, shift=shift).check()


@pytest.mark.parametrize("far", [100000, 2000000, 2 ** 31 - 6000, -2 ** 31 + 100])
@pytest.mark.parametrize("base", [1e4, 1e6])
def test_far_positions(far, base):
    # 64 bits have the angle to 2^-53 of its value: 2^31 positions, 2^-22.
    Case(64, 2, 1, 128, 128, "fp32", "fp32", "fp32", far=far, base=base).check()


def test_without_weights():
    Case(40, 3, 1, 128, 128, "bf16", "bf16", "fp32", weights=False).check()
    Case(40, 3, 1, 20, 20, "fp32", "fp32", "fp32", weights=False).check()


@pytest.mark.parametrize("d, act", [(128, "bf16"), (128, "fp32"), (20, "bf16"), (64, "bf16")])
def test_in_place(d, act):
    c = Case(33, 4, 2, d, d, act, "fp32", "fp32")
    want, (dxs, _) = c.forward(), c.backward()
    grs = binding()
    dy = [x.clone() for x in c.dy]
    grs.grs_qk_norm_backward(c.shape, ptr(dy[0]), ptr(dy[1]), ptr(c.x[0]), ptr(c.x[1]), *c.tail(), ptr(dy[0]), ptr(dy[1]), None, None, None, stream())
    c.forward(out=c.x)
    for i in range(2):
        assert torch.equal(c.x[i], want[i]) and torch.equal(dy[i], dxs[i])


def test_each_gradient_alone():
    c = Case(100, 4, 2, 128, 64, "bf16", "bf16", "fp32")
    dxs, dws = c.backward()
    for dx, dw in itertools.product((True, False), repeat=2):
        a, b = c.backward(dx, dw)
        for i in range(2):
            assert a[i] is None or torch.equal(a[i], dxs[i])
            assert b[i] is None or torch.equal(b[i], dws[i])


def test_no_tokens():
    c = Case(0, 2, 2, 16, 16)
    c.forward()
    _, dws = c.backward()
    assert bool((dws[0] == 0).all()) and bool((dws[1] == 0).all())


def test_values_that_are_not_finite_stay_in_their_head():
    c = Case(8, 4, 2, 128, 128, "fp32", "fp32", "fp32")
    c.x[0][3, 128 + 5] = float("nan")
    c.dy[1][2, 7] = float("inf")
    o, (dxs, _) = c.forward(), c.backward()
    for got, t, head, hs in ((o[0], 3, 1, 4), (dxs[0], 3, 1, 4), (dxs[1], 2, 0, 2)):
        bad = ~got.view(8, hs, 128).isfinite()
        assert bool(bad[t, head].any())
        bad[t, head] = False
        assert not bool(bad.any())
    # zeros: the norm of a head of zeros is eps alone
    c = Case(4, 2, 1, 64, 64, "bf16", "bf16", "fp32")
    c.x[0].zero_()
    assert bool((c.forward()[0] == 0).all())
    c.check()


def test_same_bits_again_and_in_a_graph():
    c = Case(3000, 8, 2, 128, 128, "bf16", "bf16", "fp32", pad=16)
    o, (dxs, dws) = c.forward(), c.backward()
    grs = binding()
    po, pdx = [torch.zeros_like(x) for x in o], [torch.full_like(x, 7.0) for x in dxs]
    pdw = [torch.zeros_like(x) for x in dws]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            c.forward(out=po)
            grs.grs_qk_norm_backward(c.shape, ptr(c.dy[0]), ptr(c.dy[1]), ptr(c.x[0]), ptr(c.x[1]), *c.tail(), ptr(pdx[0]), ptr(pdx[1]),
                                     ptr(pdw[0]), ptr(pdw[1]), ptr(c.ws), stream())
        for _ in range(2):
            graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(po + pdx + pdw, o + dxs + dws):
        assert torch.equal(a, b)


def test_gradients_are_the_differences():
    """<gradients, v> against central differences of the loss <outputs, dy>, in fp32."""
    c = Case(6, 2, 1, 48, 32, "fp32", "fp32", "fp32", pairs=True)
    dxs, dws = c.backward()
    g = torch.Generator(device="cuda").manual_seed(2)
    for grad, at in ((dxs[0], c.x[0]), (dxs[1], c.x[1]), (dws[0], c.w[0]), (dws[1], c.w[1])):
        v = torch.randn(at.shape, generator=g, device="cuda")
        old, loss, step = at.clone(), [], 2.0 ** -6
        for sign in (1, -1):
            at.copy_(old + sign * step * v)
            loss.append(float(sum((o.double() * dy.double()).sum() for o, dy in zip(c.forward(), c.dy))))
        at.copy_(old)
        want = float((grad.double() * v.double()).sum())
        # rounding: outputs of magnitude 3 to 2^-20, over the step; the third derivative's part, step^2 / 6 of like magnitudes
        size = float(sum(dy.double().abs().sum() for dy in c.dy))
        assert abs((loss[0] - loss[1]) / (2 * step) - want) <= size * (3 * 2.0 ** -20 / step + step * step)
