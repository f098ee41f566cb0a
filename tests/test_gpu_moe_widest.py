"""The widest vectors that the expert calls take, 2^30 elements: 4 GB each in fp32."""
import pytest
import torch

from test_gpu_moe import grs, stream  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act,code", [(torch.float32, 1), (torch.bfloat16, 0)])
def test_vectors_of_the_largest_width(grs, act, code):  # noqa: F811
    d = grs.GRS_MAX_WIDTH
    if torch.cuda.mem_get_info()[0] < 8 * d * act.itemsize:
        pytest.skip("needs up to 32 GB of device memory")
    s = grs.make_moe(2, 1, 4, 0, 4, d, code)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(2, d, dtype=act, device="cuda").uniform_(-1, 1, generator=g)
    xs = torch.zeros_like(x)
    rows = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    grs.grs_moe_dispatch(s, x.data_ptr(), rows.data_ptr(), xs.data_ptr(), stream())
    assert torch.equal(xs[1], x[0]) and torch.equal(xs[0], x[1])
    w = torch.tensor([0.5, 2.0], device="cuda")
    y = torch.zeros_like(x)
    grs.grs_moe_combine(s, xs.data_ptr(), rows.data_ptr(), w.data_ptr(), y.data_ptr(), stream())
    for t in (0, 1):
        assert torch.equal(y[t], x[t] * float(w[t]))
    grs.grs_moe_dispatch_backward(s, xs.data_ptr(), rows.data_ptr(), y.data_ptr(), stream())
    assert torch.equal(y, x)
    xs.fill_(0.25)  # dw is then a quarter of the sum of dy
    dys, dw = y, torch.zeros(2, device="cuda")
    grs.grs_moe_combine_backward(s, x.data_ptr(), xs.data_ptr(), rows.data_ptr(), w.data_ptr(), dys.data_ptr(), dw.data_ptr(), stream())
    for t in (0, 1):
        assert torch.equal(dys[1 - t], x[t] * float(w[t]))
    assert torch.isfinite(dw).all()
    del x, xs, y, dys
    torch.cuda.empty_cache()
