"""Refusals of the self-test of the experts' waits, before anything is launched."""
import pytest


@pytest.fixture(scope="module")
def grs():
    from gradient_reduction_sharded_gb300 import _build
    _build.build()
    from gradient_reduction_sharded_gb300 import grs as g
    return g


A = 1 << 20


@pytest.mark.parametrize("status, shape, args", [
    ("INVALID_ARG", (10, 3, 16, 8, 0, 1), (-1, 0)), ("INVALID_ARG", (10, 3, 16, 8, 0, 1), (0, -1)), ("INVALID_ARG", (10, 3, 16, 8, 1, 1), (0, 0)),
    ("SHAPE", (10, 0, 16, 8, 0, 1), (0, 0))])
def test_refusals(grs, status, shape, args):
    with pytest.raises(grs.GrsError) as e:
        grs.grs_selftest_experts_wait(grs.make_experts(*shape), A, A, A, A, A, A, A, *args, 0)
    assert e.value.status == getattr(grs, "GRS_ERR_" + status)
    assert "grs_selftest_experts_wait" in str(e.value)


def test_pointers_are_refused_as_backward_s(grs):
    s = grs.make_experts(10, 3, 16, 8, 0, 1)
    for i, off in ((0, 8), (1, 2), (5, 2), (6, 4)):
        args = [A] * 7
        args[i] += off
        with pytest.raises(grs.GrsError) as e:
            grs.grs_selftest_experts_wait(s, *args, 0, 0, 0)
        assert e.value.status == grs.GRS_ERR_ALIGNMENT
