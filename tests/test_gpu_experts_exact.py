"""Products of the experts on small whole numbers: every sum is a whole number
below 2^24, so fp32 has it exactly in any order, on the tensor cores too, and
results have to be equal to the last bit.  A lost or doubled row, feature or
slice shows, however long the sum."""
import pytest
import torch

from operators_support import DT, binding, dtype_code, ptr, stream

on_gpu = pytest.mark.gpu


def whole(shape, g, device):
    """-2, -1, 1 or 2, so that nothing that is left out is nothing."""
    x = torch.randint(-2, 2, shape, generator=g, device=device)
    return torch.where(x >= 0, x + 1, x)


class Exact:
    def __init__(self, counts, k, n, act="bf16", grad="bf16", first=0, tail=0, pad_x=0, pad_y=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(k * 7 + n)
        self.k, self.n, self.act, self.grad, self.device = k, n, act, grad, device
        self.pad_x, self.pad_y = pad_x, pad_y
        self.at = [first]
        for c in counts:
            self.at.append(self.at[-1] + c)
        self.rows = self.at[-1] + tail

        def rect(width, pad):
            m = torch.full((self.rows, width + pad), float("nan"), dtype=DT[act], device=device)
            m[first:self.at[-1], :width] = whole((self.at[-1] - first, width), g, device).to(DT[act])
            return m[:, :width]

        self.xs, self.dys = rect(k, pad_x), rect(n, pad_y)
        self.w = whole((len(counts), n, k), g, device).to(DT[act])

    def wanted(self, without=None):
        """ys, dxs and dw; `without` leaves a row out of dw's sums."""
        ys = torch.full((self.rows, self.n), 7.0, dtype=DT[self.act], device=self.device)
        dxs = torch.full((self.rows, self.k), 7.0, dtype=DT[self.act], device=self.device)
        dw = torch.zeros(self.w.shape, dtype=DT[self.grad], device=self.device)
        for e, (b, f) in enumerate(zip(self.at, self.at[1:])):
            x, d, w = self.xs[b:f].double(), self.dys[b:f].double(), self.w[e].double()
            ys[b:f] = (x @ w.T).to(ys.dtype)
            dxs[b:f] = (d @ w).to(dxs.dtype)
            if without is not None and b <= without < f:
                x[without - b] = 0
            dw[e] = (d.T @ x).to(dw.dtype)
        return ys, dxs, dw

    def check(self):
        grs = binding()
        offsets = torch.tensor(self.at, dtype=torch.int32, device="cuda")
        shape = grs.make_experts(self.rows, len(self.at) - 1, self.k, self.n, dtype_code(self.act), dtype_code(self.grad),
                                 ld_x=self.k + self.pad_x, ld_y=self.n + self.pad_y)
        size = grs.grs_experts_workspace_bytes(shape)
        ws = torch.full((max(size, 16),), 0xFF, dtype=torch.uint8, device="cuda")
        ys = torch.full((self.rows, self.n + self.pad_y), 7.0, dtype=DT[self.act], device="cuda")
        dxs = torch.full((self.rows, self.k + self.pad_x), 7.0, dtype=DT[self.act], device="cuda")
        dw = torch.full(self.w.shape, 7.0, dtype=DT[self.grad], device="cuda")
        grs.grs_experts_forward(shape, ptr(self.xs), ptr(self.w), ptr(offsets), ptr(ys), ptr(ws), stream())
        grs.grs_experts_backward(shape, ptr(self.dys), ptr(self.xs), ptr(self.w), ptr(offsets), ptr(dxs), ptr(dw), ptr(ws), stream())
        assert grs.grs_operators_check_device_errors(stream()) == grs.GRS_OK
        want = self.wanted()
        for got, name, w in ((ys[:, :self.n], "ys", want[0]), (dxs[:, :self.k], "dxs", want[1]), (dw, "dw", want[2])):
            bad = got != w
            assert not bool(bad.any()), (name, int(bad.sum()), bad.nonzero()[:4].tolist())
        assert bool((ys[:, self.n:] == 7).all()) and bool((dxs[:, self.k:] == 7).all())


@pytest.fixture(scope="module")
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


LONG = [([3], 8200, 64), ([20, 0, 1], 4100, 136), ([200], 16384, 8), ([5000, 3], 64, 40), ([20003], 8, 16), ([0, 9000, 0], 72, 24), ([100, 300], 33, 9000),
        ([1500, 4], 2056, 2056), ([4096], 2304, 2304), ([4097, 8191, 0, 8193], 768, 1032), ([20003], 776, 2056)]


@on_gpu
@pytest.mark.parametrize("counts, k, n", LONG)
@pytest.mark.parametrize("act, grad", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16")])
def test_long_sums_and_their_slices(cuda, counts, k, n, act, grad):
    Exact(counts, k, n, act, grad, first=1, tail=3).check()


# Sections of 4096 of k and what is left of them, in tiles of 16, 64, 128 and 256 rows; whole products and slices.
@on_gpu
@pytest.mark.parametrize("rows, n", [(12, 39200), (30, 39200), (100, 19600), (300, 9728), (30, 5000)])
@pytest.mark.parametrize("k", [4096, 4104, 8192, 8193 + 7, 12500])
def test_sections_of_a_long_k(cuda, rows, n, k):
    Exact([rows], k, n, tail=2).check()
    Exact([rows], n, k, tail=2).check()


@on_gpu
@pytest.mark.parametrize("counts, k, n", [([138, 6], 507, 120), ([749], 251, 1208), ([64, 65, 63], 640, 129), ([130, 0, 1, 257, 16, 127, 64], 136, 72),
                                          ([33, 160, 31, 0, 257, 300, 1, 480] * 2, 1048, 2056), ([700, 650], 2040, 72), ([70, 0, 33, 200], 1027, 519)])
@pytest.mark.parametrize("act, grad", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_ends_of_experts(cuda, counts, k, n, act, grad, pad):
    Exact(counts, k, n, act, grad, first=5, tail=40, pad_x=pad, pad_y=2 * pad).check()


# Up to eight rows in all, which forward leaves to the ordinary cores, and nine and widths that it does not: several and
# empty experts, a second group of four rows, odd numbers of results, k below a warp's 256 and beyond, rows inside wider ones.
@on_gpu
@pytest.mark.parametrize("counts", [[1], [8], [5, 0, 3], [0, 4, 0, 1, 2], [0, 0, 7, 1, 0], [1] * 8, [9], [3, 0, 6]])
@pytest.mark.parametrize("n", [1, 7, 64, 129])
@pytest.mark.parametrize("k", [8, 136, 1032, 2056, 35])
def test_a_few_rows(cuda, counts, n, k):
    Exact(counts, k, n).check()
    Exact(counts, k, n, pad_x=8, pad_y=3).check()


@on_gpu
@pytest.mark.parametrize("counts, first, tail", [([1], 3, 4), ([4, 2], 1, 1), ([0, 5, 0], 0, 3), ([2, 0, 1, 3], 2, 0), ([0, 0], 4, 4)])
@pytest.mark.parametrize("n, k, pad", [(7, 136, 0), (130, 1032, 8), (1, 8, 16)])
def test_a_few_rows_of_which_some_are_no_expert_s(cuda, counts, first, tail, n, k, pad):
    Exact(counts, k, n, first=first, tail=tail, pad_x=pad, pad_y=1).check()


@pytest.mark.parametrize("counts, k, n", [([20003], 8, 16), ([0, 9000, 0], 72, 24), ([5000, 3], 64, 40)])
@pytest.mark.parametrize("grad", ["bf16", "fp32"])
def test_one_row_left_out_would_show(counts, k, n, grad):
    """Of the sums that the tests above ask for, in 64 bits on the CPU: without any of these rows they differ."""
    c = Exact(counts, k, n, "bf16", grad, first=1, tail=3, device="cpu")
    want = c.wanted()[2]
    most = max(zip(c.at, c.at[1:]), key=lambda r: r[1] - r[0])
    for row in (most[0], most[0] + 511, most[0] + 512, (most[0] + most[1]) // 2, most[1] - 1):
        assert int((c.wanted(without=row)[2] != want).sum()) > 10
