"""Shapes whose elements no memory holds: refused, where their bytes would not
fit 64 bits and the answers would be of another shape."""
import pytest


@pytest.fixture(scope="module")
def grs():
    from gradient_reduction_sharded_gb300 import _build
    _build.build()
    from gradient_reduction_sharded_gb300 import grs as g
    return g


A = 1 << 20
WIDE = 1 << 30


def refused(grs, call, *args, status="SHAPE"):
    with pytest.raises(grs.GrsError) as e:
        call(*args)
    assert e.value.status == getattr(grs, "GRS_ERR_" + status), e.value


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("rows, experts, k, n, ld_x, ld_y", [
    (0, 1024, WIDE, WIDE, 0, 0), (1000, 1024, WIDE, WIDE, 0, 0), (5, 1024, WIDE - 1, WIDE - 1, 0, 0), (10, 1, WIDE, 1025, 0, 0),
    ((1 << 31) - (1 << 16), 1, 8, 8, WIDE, 0), ((1 << 31) - (1 << 16), 1, 8, 8, 0, WIDE), ((1 << 31) - (1 << 16), 1, 1025, 8, 0, 0)])
def test_experts(grs, dtype, rows, experts, k, n, ld_x, ld_y):
    s = grs.make_experts(rows, experts, k, n, dtype, 1, ld_x, ld_y)
    refused(grs, grs.grs_experts_workspace_bytes, s, status="INVALID_ARG")
    refused(grs, grs.grs_experts_forward, s, A, A, A, A, A, 0)
    refused(grs, grs.grs_experts_backward, s, A, A, A, A, A, A, A, 0)


@pytest.mark.parametrize("rows, experts, k, n", [(1 << 30, 1, 1024, 8), (10, 1024, 1 << 15, 1 << 15), (3, 1, WIDE, 1024)])
def test_experts_up_to_the_limit_have_a_workspace(grs, rows, experts, k, n):
    for dtype in (0, 1):
        assert grs.grs_experts_workspace_bytes(grs.make_experts(rows, experts, k, n, dtype, 1)) >= 0
    # Of rows that are not whole 16-byte chunks: copies of all of them.
    assert grs.grs_experts_workspace_bytes(grs.make_experts(rows // 2, experts, k - 1, n, 0, 1)) >= 2 * (rows // 2 + experts * n) * k


@pytest.mark.parametrize("tokens, q, k, d, ld", [
    (1 << 40, WIDE, 0, 1, (0, 0, 0, 0)), (1 << 40, 0, 1 << 23, 1, (0, 0, 0, 0)), (1 << 40, 1, 1, 1, (0, 0, 0, 0)), (1 << 39, 1 << 20, 0, 1024, (0, 0, 0, 0)),
    (1 << 30, 1, 1, 8, (1 << 11, 0, 0, 0)), (1 << 30, 1, 1, 8, (0, 0, 0, 1 << 11))])
def test_qk_norm(grs, tokens, q, k, d, ld):
    s = grs.make_qk_norm(tokens, q, k, d, 0, 1e-6, 0, 0, 0, False, *ld)
    refused(grs, grs.grs_qk_norm_workspace_bytes, s, status="INVALID_ARG")
    refused(grs, grs.grs_qk_norm_forward, s, *[A] * 8, 0)
    refused(grs, grs.grs_qk_norm_backward, s, *[A] * 13, 0)


def test_qk_norm_of_many_tokens_has_a_workspace(grs):
    assert grs.grs_qk_norm_workspace_bytes(grs.make_qk_norm(1 << 33, 64, 64, 1, 0, 1e-6, 0, 0, 0)) > 0
    assert grs.grs_qk_norm_workspace_bytes(grs.make_qk_norm(1, 2, 2, 64, 0, 1e-6, 0, 0, 0, ld_q=1 << 40)) > 0
