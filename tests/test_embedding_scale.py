"""The embedding's scale has to be a number: padding and rows without tokens are
zeros, which infinity or NaN times zero is not."""
import math

import pytest
import torch


@pytest.fixture(scope="module")
def grs():
    from gradient_reduction_sharded_gb300 import _build
    _build.build()
    from gradient_reduction_sharded_gb300 import grs as g
    return g


A = 1 << 20


@pytest.mark.parametrize("scale", [math.inf, -math.inf, math.nan])
def test_a_scale_that_is_not_finite_is_refused(grs, scale):
    s = grs.make_embedding(5, 0, 20, 16, scale, 0, 0)
    for call, args in ((grs.grs_embedding_workspace_bytes, (s,)), (grs.grs_embedding_forward, (s, A, A, A, 0)), (grs.grs_embedding_backward, (s, A, A, A, A, 0))):
        with pytest.raises(grs.GrsError) as e:
            call(*args)
        assert e.value.status == grs.GRS_ERR_INVALID_ARG
    assert "scale" in str(e.value)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [torch.finfo(torch.float32).max, 2.0 ** -140, -3.0, 0.0])
def test_padding_is_zero_at_any_finite_scale(grs, scale):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    ids = torch.tensor([3, -1, 0, 99, 3], dtype=torch.int32, device="cuda")
    table, y, dtable = (torch.full(n, 7.0, device="cuda") for n in ((10, 16), (5, 16), (10, 16)))
    s = grs.make_embedding(5, 0, 10, 16, scale, grs.GRS_DTYPE_FP32, grs.GRS_DTYPE_FP32)
    ws = torch.empty(grs.grs_embedding_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    grs.grs_embedding_forward(s, ids.data_ptr(), table.data_ptr(), y.data_ptr(), st)
    assert bool((y[[1, 3]] == 0).all())
    dy = torch.ones(5, 16, device="cuda")
    grs.grs_embedding_backward(s, ids.data_ptr(), dy.data_ptr(), dtable.data_ptr(), ws.data_ptr(), st)
    assert bool((dtable[[1, 2, 4, 5, 6, 7, 8, 9]] == 0).all())
