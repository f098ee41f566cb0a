"""Embedding and its table's gradient against 64 bits: parts of a vocabulary,
ids of no row, ids that fill a batch, vectors of any size and alignment."""
import pytest
import torch

from operators_support import DT, binding, close, dtype_code, half, ptr, stream

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def at(shape, dtype, shift):
    """An uninitialised matrix `shift` elements after a 16-byte boundary, 9s around it."""
    n = shape[0] * shape[1]
    wide = torch.full((n + 32,), 9.0, dtype=dtype, device="cuda")
    return wide, wide[8 + shift:8 + shift + n].view(shape)


def run(ids, begin, end, d, act, grad, scale, shift=0, seed=0):
    grs = binding()
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = ids.numel()
    shape = grs.make_embedding(t, begin, end, d, scale, dtype_code(act), dtype_code(grad))
    scale = torch.tensor(scale, dtype=torch.float32).item()
    row = ids.long() - begin
    held = (row >= 0) & (row < end - begin)
    _, table = at((end - begin, d), DT[act], shift)
    table.copy_(torch.randn(end - begin, d, generator=g, device="cuda"))
    wide, y = at((t, d), DT[act], shift)
    grs.grs_embedding_forward(shape, ptr(ids), ptr(table), ptr(y), stream())
    want = torch.zeros(t, d, dtype=torch.float64, device="cuda")
    want[held] = table.double()[row[held]] * scale
    # one product in fp32, one rounding to the type
    close(y, want, want.abs() * (2.0 ** -24 + half(act)) * 1.01, "y")
    assert bool((wide[:8 + shift] == 9).all()) and bool((wide[8 + shift + t * d:] == 9).all())

    _, dy = at((t, d), DT[act], shift)
    dy.copy_(torch.randn(t, d, generator=g, device="cuda"))
    wide, dt = at((end - begin, d), DT[grad], shift)
    ws = torch.full((max(16, grs.grs_embedding_workspace_bytes(shape)),), 0xFF, dtype=torch.uint8, device="cuda")
    grs.grs_embedding_backward(shape, ptr(ids), ptr(dy), ptr(dt), ptr(ws), stream())
    assert grs.grs_operators_check_device_errors(stream()) == grs.GRS_OK
    want = torch.zeros(end - begin, d, dtype=torch.float64, device="cuda").index_add_(0, row[held], dy[held].double()) * scale
    size = torch.zeros_like(want).index_add_(0, row[held], dy[held].double().abs()) * scale
    n = torch.zeros(end - begin, dtype=torch.float64, device="cuda").index_add_(0, row[held], torch.ones_like(row[held], dtype=torch.float64))
    # n - 1 additions, one product, one rounding to the type
    close(dt, want, size * n[:, None] * 2.0 ** -24 + want.abs() * half(grad) * 1.01, "dtable")
    assert bool((wide[:8 + shift] == 9).all()) and bool((wide[8 + shift + want.numel():] == 9).all())
    return dt, ws, shape, dy


def tokens(n, lo, hi, seed=0):
    return torch.randint(lo, hi, (n,), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda", dtype=torch.int32)


@pytest.mark.parametrize("act, grad", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("d, shift", [(64, 0), (8, 0), (1, 0), (519, 0), (64, 1), (2048, 0), (776, 2)])
def test_sizes_and_types(d, shift, act, grad):
    run(tokens(300, -3, 120), 7, 101, d, act, grad, 1.7, shift)


@pytest.mark.parametrize("n", [1, 31, 32, 33, 1024, 1025, 5000, 40000])
@pytest.mark.parametrize("vocab", [1, 2, 511, 512, 151936])
def test_numbers_of_tokens_and_rows(n, vocab):
    run(tokens(n, 0, vocab, seed=n), 0, vocab, 16, "bf16", "fp32", 1.0)


@pytest.mark.parametrize("n", [200, 4096, 30000])
def test_ids_that_fill_a_batch(n):
    ids = tokens(n, 0, 50)
    ids[torch.rand(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) < 0.6] = 17
    run(ids, 0, 50, 72, "fp32", "fp32", 2.0)
    ids[: n // 2] = -1
    run(ids, 17, 30, 72, "bf16", "bf16", 0.5)
    run(torch.full((n,), 3, dtype=torch.int32, device="cuda"), 0, 5, 40, "bf16", "fp32", 1.0)
    run(torch.full((n,), -1, dtype=torch.int32, device="cuda"), 0, 5, 40, "bf16", "bf16", 1.0)


def test_ids_at_the_ends_of_their_type():
    ids = torch.tensor([-2 ** 31, 2 ** 31 - 1, 2 ** 31 - 2, 0, -1, 2 ** 31 - 8], dtype=torch.int32, device="cuda")
    run(ids, 2 ** 31 - 9, 2 ** 31 - 1, 16, "fp32", "fp32", 1.0)
    run(ids, 0, 4, 16, "fp32", "fp32", 1.0)


def test_many_tokens_of_a_few_rows():
    run(tokens(300000, 0, 3), 0, 3, 8, "bf16", "fp32", 1.0)


def test_a_large_vocabulary_of_short_vectors():
    run(tokens(700000, 0, 1 << 20), 0, 1 << 20, 8, "fp32", "fp32", 1.0)


def test_values_that_are_not_finite_stay_in_their_row():
    grs = binding()
    ids = torch.tensor([4, 1, 4, -1, 2], dtype=torch.int32, device="cuda")
    dy = torch.ones(5, 16, device="cuda")
    dy[2], dy[3] = float("inf"), float("nan")
    shape = grs.make_embedding(5, 0, 6, 16, 1.0, grs.GRS_DTYPE_FP32, grs.GRS_DTYPE_FP32)
    ws = torch.empty(grs.grs_embedding_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
    dt = torch.empty(6, 16, device="cuda")
    grs.grs_embedding_backward(shape, ptr(ids), ptr(dy), ptr(dt), ptr(ws), stream())
    assert bool((dt[4] == float("inf")).all()) and dt[[0, 1, 2, 3, 5], 0].tolist() == [0, 1, 1, 0, 0]


def test_no_tokens_clear_the_gradient():
    grs = binding()
    shape = grs.make_embedding(0, 0, 6, 5, 1.0, grs.GRS_DTYPE_BF16, grs.GRS_DTYPE_BF16)
    dt = torch.ones(6, 5, dtype=torch.bfloat16, device="cuda")
    grs.grs_embedding_backward(shape, None, None, ptr(dt), None, stream())
    assert bool((dt == 0).all())


def test_same_bits_again_and_in_a_graph():
    grs = binding()
    ids = tokens(20000, -5, 3000, seed=2)
    ids[:6000] = 11
    dt, ws, shape, dy = run(ids, 0, 2990, 264, "bf16", "fp32", 3.0)
    out = torch.empty_like(dt)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            grs.grs_embedding_backward(shape, ptr(ids), ptr(dy), ptr(out), ptr(ws), stream())
        for _ in range(3):
            ws.fill_(0xFF)
            out.zero_()
            graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, dt)
