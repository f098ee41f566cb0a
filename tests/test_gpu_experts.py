"""Products of the experts against 64 bits: every type, ragged and empty
experts, rows that are no expert's, distances of rows, widths that divide
nothing."""
import pytest
import torch

from operators_support import DT, binding, close, dtype_code, half, ptr, stream

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def chain(k):
    """Error of a sum of k products in fp32, of the sum of their magnitudes, whatever the order
    and however each of at most k additions is rounded (2^-23: towards zero)."""
    return k * 2.0 ** -23


class Case:
    def __init__(self, counts, k, n, act="bf16", grad="bf16", first=0, tail=0, pad_x=0, pad_y=0, seed=0, mean=0.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.k, self.n, self.act, self.grad, self.counts = k, n, act, grad, counts
        at = [first]
        for c in counts:
            at.append(at[-1] + c)
        self.at, self.rows = at, at[-1] + tail
        self.offsets = torch.tensor(at, dtype=torch.int32, device="cuda")
        self.pad_x, self.pad_y = pad_x, pad_y
        dt = DT[act]

        def rect(width, pad, std):
            wide = torch.full((self.rows, width + pad), float("nan"), dtype=dt, device="cuda")
            wide[first:at[-1], :width] = torch.randn(at[-1] - first, width, generator=g, device="cuda").mul_(std).add_(mean)
            return wide[:, :width]  # what is no expert's is NaN

        self.xs, self.dys = rect(k, pad_x, 1.0), rect(n, pad_y, 0.1)
        self.w = (torch.randn(len(counts), n, k, generator=g, device="cuda") * k ** -0.5).to(dt)
        grs = binding()
        self.shape = grs.make_experts(self.rows, len(counts), k, n, dtype_code(act), dtype_code(grad), ld_x=k + pad_x, ld_y=n + pad_y)
        size = grs.grs_experts_workspace_bytes(self.shape)
        self.ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") if size else None

    def out(self, width, pad):
        return torch.full((self.rows, width + pad), 7.0, dtype=DT[self.act], device="cuda")

    def forward(self):
        ys = self.out(self.n, self.pad_y)
        binding().grs_experts_forward(self.shape, ptr(self.xs), ptr(self.w), ptr(self.offsets), ptr(ys), ptr(self.ws), stream())
        return ys

    def backward(self, rows=True, weights=True):
        dxs = self.out(self.k, self.pad_x) if rows else None
        dw = torch.full(self.w.shape, 7.0, dtype=DT[self.grad], device="cuda") if weights else None
        binding().grs_experts_backward(self.shape, ptr(self.dys), ptr(self.xs) if weights else None, ptr(self.w) if rows else None,
                                       ptr(self.offsets), ptr(dxs), ptr(dw), ptr(self.ws), stream())
        return dxs, dw

    def check_rows(self, got, a, of, width, terms, what):
        """got[r] = a[r] @ of(w[e]) over the experts' rows, the rest as it was."""
        assert bool((got[:self.at[0]] == 7).all()) and bool((got[self.at[-1]:] == 7).all()), what
        assert bool((got[:, width:] == 7).all()), what
        for e, (b, f) in enumerate(zip(self.at, self.at[1:])):
            m = of(self.w[e].double())
            x = a[b:f].double()
            want = x @ m
            close(got[b:f, :width], want, (x.abs() @ m.abs()) * chain(terms) + want.abs() * half(self.act), (what, e))

    def check(self):
        ys = self.forward()
        dxs, dw = self.backward()
        assert binding().grs_operators_check_device_errors(stream()) == binding().GRS_OK
        self.check_rows(ys, self.xs, lambda m: m.T, self.n, self.k, "ys")
        self.check_rows(dxs, self.dys, lambda m: m, self.k, self.n, "dxs")
        for e, (b, f) in enumerate(zip(self.at, self.at[1:])):
            d, x = self.dys[b:f].double(), self.xs[b:f].double()
            want = d.T @ x
            close(dw[e], want, (d.T.abs() @ x.abs()) * chain(f - b) + want.abs() * half(self.grad), ("dw", e))


COUNTS = {"one": [1], "few": [3, 0, 1, 2], "ragged": [130, 0, 1, 257, 16, 127, 64], "even": [256, 256], "none": [0, 0, 0]}


@pytest.mark.parametrize("act, grad", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("counts", sorted(COUNTS))
def test_ragged_experts(counts, act, grad):
    Case(COUNTS[counts], 136, 72, act, grad, first=3, tail=5).check()


@pytest.mark.parametrize("k, n", [(8, 8), (1, 1), (64, 128), (128, 64), (192, 520), (520, 200), (1000, 264), (1027, 519), (33, 300), (2048, 16)])
@pytest.mark.parametrize("act", ["bf16", "fp32"])
def test_widths(k, n, act):
    Case([70, 0, 33, 200], k, n, act, "fp32", tail=9).check()


@pytest.mark.parametrize("pad_x, pad_y", [(8, 64), (3, 0), (0, 5), (16, 1)])
@pytest.mark.parametrize("act", ["bf16", "fp32"])
def test_rows_inside_wider_ones(pad_x, pad_y, act):
    Case([50, 300, 1], 200, 136, act, "bf16", first=2, tail=130, pad_x=pad_x, pad_y=pad_y).check()


def test_many_experts():
    g = torch.Generator().manual_seed(3)
    Case(torch.randint(0, 9, (1024,), generator=g).tolist(), 72, 136, "bf16", "bf16").check()


def test_a_large_expert_beside_small_ones():
    Case([5, 4097, 11, 0, 700], 776, 1032, "bf16", "fp32", tail=77).check()


@pytest.mark.parametrize("counts, k, n", [([3], 8200, 64), ([20, 0, 1], 4100, 136), ([200], 16384, 8), ([5000, 3], 64, 40), ([20003], 8, 16),
                                          ([0, 9000, 0], 72, 24), ([100, 300], 33, 9000), ([1500, 4], 2056, 2056)])
@pytest.mark.parametrize("act, grad", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16")])
def test_a_long_k_with_few_tiles(counts, k, n, act, grad):
    Case(counts, k, n, act, grad, first=1, tail=3).check()


@pytest.mark.parametrize("counts, k, n", [([138, 6], 507, 120), ([1, 0, 0], 1300, 123), ([749], 251, 1208), ([64, 65, 63], 640, 129), ([90, 0, 7], 65, 64)])
@pytest.mark.parametrize("act, grad", [("fp32", "fp32"), ("fp32", "bf16")])
def test_fp32_in_slices(counts, k, n, act, grad):
    Case(counts, k, n, act, grad, first=2, tail=1).check()


@pytest.mark.parametrize("counts, k, n", [([33, 160, 31, 0, 257, 300, 1, 480] * 2, 1048, 2056), ([95, 97, 0, 64, 130], 136, 264), ([700, 650], 2040, 72)])
@pytest.mark.parametrize("pad", [0, 8, 4])
def test_ends_of_experts_and_of_rows_inside_a_box_of_results(counts, k, n, pad):
    Case(counts, k, n, "bf16", "bf16", first=5, tail=40, pad_x=pad, pad_y=2 * pad).check()


@pytest.mark.parametrize("experts, k, n", [(81, 152, 340), (400, 264, 296), (400, 260, 33), (90, 131, 300)])
@pytest.mark.parametrize("grad", ["bf16", "fp32"])
def test_weights_of_experts_without_rows_have_no_gradient(experts, k, n, grad):
    counts = [0] * experts
    counts[3], counts[experts // 2], counts[-2] = 5, 1, 17
    Case(counts, k, n, "bf16", grad, tail=2).check()


def test_offsets_outside_the_rows_are_taken_as_the_nearest():
    c = Case([40, 20, 30], 64, 64)
    want = c.forward()
    c.offsets[3] = 1000
    c.offsets[0] = -5
    assert torch.equal(c.forward(), want)


def test_one_of_the_gradients():
    c = Case([100, 30], 264, 128)
    both = c.backward()
    assert torch.equal(c.backward(weights=False)[0], both[0])
    assert torch.equal(c.backward(rows=False)[1], both[1])


def test_no_rows_clear_the_weights_gradient():
    c = Case([0, 0], 24, 40, tail=0)
    dxs, dw = c.backward()
    assert bool((dw == 0).all())


def test_infinities_stay_with_their_rows():
    c = Case([30, 40], 128, 128)
    c.xs[10, 5] = float("inf")
    c.dys[12, 3] = float("nan")
    ys = c.forward()
    dxs, dw = c.backward()
    fine = torch.ones(70, dtype=torch.bool, device="cuda")
    fine[10] = False
    assert bool(ys[fine].isfinite().all()) and not bool(ys[10].isfinite().any())
    fine[10], fine[12] = True, False
    assert bool(dxs[fine].isfinite().all()) and bool(dxs[12].isnan().all())
    assert bool(dw[1].isfinite().all())
    assert not bool(dw[0][3].isfinite().any()) and not bool(dw[0][:, 5].isfinite().any())


def test_same_bits_again_and_in_a_graph_on_another_stream():
    c = Case([300, 0, 1000, 17], 512, 264, "bf16", "fp32", tail=4)
    ys, (dxs, dw) = c.forward(), c.backward()
    out = [c.out(c.n, 0), c.out(c.k, 0), torch.full_like(dw, 7.0)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    grs = binding()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            grs.grs_experts_forward(c.shape, ptr(c.xs), ptr(c.w), ptr(c.offsets), ptr(out[0]), ptr(c.ws), stream())
            grs.grs_experts_backward(c.shape, ptr(c.dys), ptr(c.xs), ptr(c.w), ptr(c.offsets), ptr(out[1]), ptr(out[2]), ptr(c.ws), stream())
        for _ in range(2):
            graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, (ys, dxs, dw)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # Other row counts under the same graph: the offsets are read at the replay.
    d = Case([5, 800, 20, 490], 512, 264, "bf16", "fp32", tail=6, seed=1)
    c.offsets.copy_(d.offsets)
    c.xs.copy_(d.xs)
    c.dys.copy_(d.dys)
    c.w.copy_(d.w)
    want = d.forward(), *d.backward()
    for t in out:
        t.fill_(7.0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_gradients_are_the_differences():
    """<dxs, v> and <dw, v> against the change of the loss <ys, dys> along v, in fp32."""
    c = Case([20, 0, 33], 48, 40, "fp32", "fp32")
    grs = binding()
    dxs, dw = c.backward()
    g = torch.Generator(device="cuda").manual_seed(9)
    for grad, at in ((dxs, c.xs), (dw, c.w)):
        v = torch.randn(at.shape, generator=g, device="cuda")
        old, loss = at.clone(), []
        for sign in (1, -1):
            at.copy_(old + sign * 0.5 * v)
            loss.append(float((c.forward().double() * c.dys.double()).sum()))
        at.copy_(old)
        # The map is linear in each of the two, so the difference has no error of its own: fp32 chains of 48 products
        # and the rounding of old +- v / 2, of terms whose magnitudes add up to `size`.
        size = float((grad.double().abs() * (v.double().abs() + 2 * old.double().abs())).sum()) + sum(abs(x) for x in loss)
        want = float((grad.double() * v.double()).sum())
        scale = float((c.dys.double().abs().sum()) * 60)
        assert abs((loss[0] - loss[1]) - want) <= 2.0 ** -22 * 64 * (size + scale)


def test_fp32_gradients_of_many_rows_are_summed_in_fp32():
    """Values of one sign, where additions that round towards zero would show: 64 bits to 2e-6 of the result."""
    c = Case([9000, 4100], 256, 128, "bf16", "fp32", mean=1.0)
    _, dw = c.backward(rows=False)
    for e, (b, f) in enumerate(zip(c.at, c.at[1:])):
        want = c.dys[b:f].double().T @ c.xs[b:f].double()
        assert float((dw[e].double() - want).norm() / want.norm()) < 2e-6
