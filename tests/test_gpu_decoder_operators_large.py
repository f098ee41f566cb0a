"""Experts' products, embedding and query and key norms on more than 2^31
elements: what lies at their ends."""
import pytest
import torch

from operators_support import binding, close, half, ptr, stream

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs up to 60 GB of device memory")
    yield
    torch.cuda.empty_cache()


def workspace(n):
    return torch.empty(max(16, n), dtype=torch.uint8, device="cuda")


def randn(*shape, seed=0, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") * std).bfloat16()


@pytest.mark.parametrize("k", [1024, 1027])
def test_rows_of_the_experts(k):
    grs = binding()
    rows, n, tail = (1 << 31) // k + 300, 64, 200
    xs, dys = torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda"), torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    xs[-tail:], dys[-tail:] = randn(tail, k), randn(tail, n, seed=1)
    w = randn(2, n, k, seed=2, std=k ** -0.5)
    off = torch.tensor([0, 1000, rows], dtype=torch.int32, device="cuda")
    s = grs.make_experts(rows, 2, k, n, grs.GRS_DTYPE_BF16, grs.GRS_DTYPE_FP32)
    ws = workspace(grs.grs_experts_workspace_bytes(s))
    ys, dxs, dw = torch.ones_like(dys), torch.ones_like(xs), torch.ones(2, n, k, device="cuda")
    grs.grs_experts_forward(s, ptr(xs), ptr(w), ptr(off), ptr(ys), ptr(ws), stream())
    grs.grs_experts_backward(s, ptr(dys), ptr(xs), ptr(w), ptr(off), ptr(dxs), ptr(dw), ptr(ws), stream())
    x, dy, m = xs[-tail:].double(), dys[-tail:].double(), w[1].double()
    for got, want, size, terms in ((ys[-tail:], x @ m.T, x.abs() @ m.abs().T, k), (dxs[-tail:], dy @ m, dy.abs() @ m.abs(), n)):
        close(got, want, size * terms * 2.0 ** -23 + want.abs() * half("bf16"), "rows")
    close(dw[1], dy.T @ x, (dy.T.abs() @ x.abs()) * tail * 2.0 ** -23, "dw")
    assert not bool(ys[:-tail].any()) and not bool(dxs[:-tail].any()) and not bool(dw[0].any())


def test_weights_of_the_experts():
    grs = binding()
    e, k, n, rows = 33, 8192, 8192, 40
    w = torch.zeros(e, n, k, dtype=torch.bfloat16, device="cuda")
    w[-1] = randn(n, k, std=k ** -0.5)
    xs, dys = randn(rows, k, seed=1), randn(rows, n, seed=2)
    off = torch.tensor([0] * e + [rows], dtype=torch.int32, device="cuda")
    s = grs.make_experts(rows, e, k, n, grs.GRS_DTYPE_BF16, grs.GRS_DTYPE_BF16)
    ws = workspace(grs.grs_experts_workspace_bytes(s))
    ys, dxs, dw = torch.ones_like(dys), torch.ones_like(xs), torch.ones_like(w)
    grs.grs_experts_forward(s, ptr(xs), ptr(w), ptr(off), ptr(ys), ptr(ws), stream())
    grs.grs_experts_backward(s, ptr(dys), ptr(xs), ptr(w), ptr(off), ptr(dxs), ptr(dw), ptr(ws), stream())
    x, dy, m = xs.double(), dys.double(), w[-1].double()
    close(ys, x @ m.T, (x.abs() @ m.abs().T) * k * 2.0 ** -23 + (x @ m.T).abs() * half("bf16"), "ys")
    close(dxs, dy @ m, (dy.abs() @ m.abs()) * n * 2.0 ** -23 + (dy @ m).abs() * half("bf16"), "dxs")
    close(dw[-1], dy.T @ x, (dy.T.abs() @ x.abs()) * rows * 2.0 ** -23 + (dy.T @ x).abs() * half("bf16"), "dw")
    assert not bool(dw[:-1].any())


@pytest.mark.parametrize("d", [2048, 2051])
def test_table(d):
    grs = binding()
    rows, t = (1 << 31) // d + 100, 3000
    table = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda")
    table[-50:] = randn(50, d)
    ids = torch.randint(rows - 50, rows, (t,), dtype=torch.int32, device="cuda")
    s = grs.make_embedding(t, 0, rows, d, 2.0, grs.GRS_DTYPE_BF16, grs.GRS_DTYPE_FP32)
    y, dy = torch.empty(t, d, dtype=torch.bfloat16, device="cuda"), randn(t, d, seed=1)
    dt = torch.ones(rows, d, device="cuda")
    ws = workspace(grs.grs_embedding_workspace_bytes(s))
    grs.grs_embedding_forward(s, ptr(ids), ptr(table), ptr(y), stream())
    grs.grs_embedding_backward(s, ptr(ids), ptr(dy), ptr(dt), ptr(ws), stream())
    assert torch.equal(y, (table[ids.long()].float() * 2).bfloat16())
    at = ids.long() - (rows - 50)
    want = torch.zeros(50, d, dtype=torch.float64, device="cuda").index_add_(0, at, dy.double()) * 2
    size = torch.zeros(50, d, dtype=torch.float64, device="cuda").index_add_(0, at, dy.double().abs()) * 2
    close(dt[-50:], want, size * t * 2.0 ** -24, "dtable")
    assert not bool(dt[:-50].any())


@pytest.mark.parametrize("d, wide", [(128, 4096), (80, 4100)])
def test_tokens_of_the_norms(d, wide):
    grs = binding()
    heads, tail = 4, 30
    t = (1 << 31) // wide + 100
    joint = torch.zeros(t, wide, dtype=torch.bfloat16, device="cuda")
    joint[-tail:] = randn(tail, wide)
    dy = torch.zeros(t, heads * d, dtype=torch.bfloat16, device="cuda")
    dy[-tail:] = randn(tail, heads * d, seed=1)
    pos = torch.arange(t, dtype=torch.int32, device="cuda")
    turns = torch.tensor(grs.grs_rope_turns([1e4 ** (-2 * i / d) for i in range(d // 2)]), dtype=torch.uint64, device="cuda")

    def run(x, g, p, ld):
        n = x.shape[0]
        s = grs.make_qk_norm(n, heads, 0, d, d, 1e-6, grs.GRS_DTYPE_BF16, grs.GRS_DTYPE_FP32, grs.GRS_DTYPE_FP32, ld_q=ld)
        ws = workspace(grs.grs_qk_norm_workspace_bytes(s))
        o, dx, dw = torch.empty_like(g), torch.zeros_like(x), torch.empty(d, device="cuda")
        grs.grs_qk_norm_forward(s, ptr(x), None, None, None, ptr(p), ptr(turns), ptr(o), None, stream())
        grs.grs_qk_norm_backward(s, ptr(g), None, ptr(x), None, None, None, ptr(p), ptr(turns), ptr(dx), None, ptr(dw), None, ptr(ws), stream())
        return o[-tail:].clone(), dx[-tail:].clone(), dw

    # The last tokens by themselves: a head's result does not depend on where it lies; the sums have another order.
    o, dx, dw = run(joint, dy, pos, wide)
    o2, dx2, dw2 = run(joint[-tail:].clone(), dy[-tail:].clone(), pos[-tail:].clone(), wide)
    assert torch.equal(o, o2) and torch.equal(dx, dx2)
    close(dw, dw2.double(), dw2.abs().double() * 0 + 2.0 ** -20 * tail * heads * 20, "dw")
