"""Long sums of the experts' products whose results leave in bf16: values of one
sign, where additions that round towards zero add up to a bias.  A single
result is within its rounding all the same, so the mean of the relative errors
of all results is what is looked at."""
import pytest
import torch

from operators_support import binding, dtype_code, half, ptr, stream

pytestmark = pytest.mark.gpu

LONG = 131072


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def limit(n):
    """Of the mean relative error of n results.  The tensor cores add 16 products an instruction and lose at most a unit
    of fp32 (2^-23) where they do; 4096 of k a section make 256 of them.  The at most 64 sections' additions lose half a
    unit each.  The results' own roundings are even on both sides: at most 2^-8, so 2^-8 / sqrt(3 n) in the mean, six times."""
    return 256 * 2.0 ** -23 + 64 * 2.0 ** -24 + 6 * half("bf16") / (3 * n) ** 0.5


def positive(rows, width, along, g):
    """Numbers in (0, 2), rows (along 0) or columns (1) scaled by factors in [0.5, 1): results spread over binades."""
    m = torch.rand(rows, width, generator=g, device="cuda") * 2
    f = torch.rand(rows if along == 0 else width, generator=g, device="cuda") * 0.5 + 0.5
    return (m * (f[:, None] if along == 0 else f)).to(torch.bfloat16)


def mean_error(got, a, b):
    """Of got against a^T b in 64 bits, a [k, m] and b [k, n] in any strides, a few columns of b at a time."""
    total, step = 0.0, max(1, 2 ** 28 // a.shape[0])
    left = a.double().T
    for c in range(0, b.shape[1], step):
        want = left @ b[:, c:c + step].double()
        total += float(((got[:, c:c + step].double() - want) / want).sum())
    return total / got.numel()


# One expert: 96 tiles of 128 x 128, and 81 of 256 x 256, so that none is cut into slices.
@pytest.mark.parametrize("k, n", [(768, 2048), (2304, 2300)])
def test_weights_gradients_of_many_rows(k, n):
    grs, g = binding(), torch.Generator(device="cuda").manual_seed(k)
    xs, dys = positive(LONG, k, 1, g), positive(LONG, n, 1, g)
    offsets = torch.tensor([0, LONG], dtype=torch.int32, device="cuda")
    shape = grs.make_experts(LONG, 1, k, n, dtype_code("bf16"), dtype_code("bf16"))
    ws = torch.empty(max(16, grs.grs_experts_workspace_bytes(shape)), dtype=torch.uint8, device="cuda")
    dw = torch.empty(n, k, dtype=torch.bfloat16, device="cuda")
    grs.grs_experts_backward(shape, ptr(dys), ptr(xs), None, ptr(offsets), None, ptr(dw), ptr(ws), stream())
    off = mean_error(dw, dys, xs)
    assert abs(off) <= limit(dw.numel()), off


# Few and many rows, whole products and (10000) ones of a few slices.
@pytest.mark.parametrize("rows, n", [(12, 39200), (30, 39200), (30, 10000), (100, 19600), (300, 9728)])
def test_rows_of_a_long_k(rows, n):
    grs, g = binding(), torch.Generator(device="cuda").manual_seed(rows + n)
    offsets = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    a, w = positive(rows, LONG, 0, g), positive(n, LONG, 0, g)
    out = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    # Forward: k is the input features; rows' gradients: the output features, across which the weights lie.
    for forward in (True, False):
        shape = grs.make_experts(rows, 1, *((LONG, n) if forward else (n, LONG)), dtype_code("bf16"), dtype_code("bf16"))
        ws = torch.empty(max(16, grs.grs_experts_workspace_bytes(shape)), dtype=torch.uint8, device="cuda")
        if forward:
            grs.grs_experts_forward(shape, ptr(a), ptr(w), ptr(offsets), ptr(out), ptr(ws), stream())
        else:
            across = w.T.contiguous()
            grs.grs_experts_backward(shape, ptr(a), None, ptr(across), ptr(offsets), ptr(out), None, ptr(ws), stream())
        off = mean_error(out, a.T, w.T)
        assert abs(off) <= limit(out.numel()), (forward, off)
        out.fill_(7)
