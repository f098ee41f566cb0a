"""Lists of separate tensors (grs_tensors_*) on the host: layout and
refusals, no GPU."""
import pytest


@pytest.fixture(scope="module")
def grs():
    from gradient_reduction_sharded_gb300 import _build
    _build.build()
    from gradient_reduction_sharded_gb300 import grs as g
    return g


def test_layout_rounds_every_tensor_up_to_a_block(grs):
    numels = [1, 0, 256, 257, 5 << 31, 300]
    h = grs.grs_tensors_create(numels, grs.GRS_PLAN_HOST_ONLY)
    try:
        want, at = [], 0
        for n in numels:
            want.append(at)
            at += -(-n // 256) * 256
        assert [grs.grs_tensors_offset(h, i) for i in range(len(numels))] == want
        info = grs.grs_tensors_query(h)
        assert info["n_tensors"] == len(numels) and info["device"] == -1
        assert info["n_elements"] == sum(numels)
        assert info["n_state"] == at and info["n_blocks"] == at // 256
        assert info["workspace_bytes"] > 0
    finally:
        grs.grs_tensors_destroy(h)


@pytest.mark.parametrize("numels,flags,status", [
    ([], 1, "GRS_ERR_INVALID_ARG"),
    ([4, -1], 1, "GRS_ERR_SHAPE"),
    ([1 << 62], 1, "GRS_ERR_SHAPE"),
    ([1 << 41, 1 << 41, 1 << 41], 1, "GRS_ERR_SHAPE"),
    ([4], 2, "GRS_ERR_INVALID_ARG"),
    ([4], 5, "GRS_ERR_INVALID_ARG"),
])
def test_create_refuses(grs, numels, flags, status):
    with pytest.raises(grs.GrsError) as e:
        grs.grs_tensors_create(numels, flags)
    assert e.value.status == getattr(grs, status) and grs.grs_last_error()


def test_host_only_lists_refuse_launches(grs):
    h = grs.grs_tensors_create([10], grs.GRS_PLAN_HOST_ONLY)
    hp = grs.make_adamw(1e-3, 0.9, 0.999, 1e-8, 0.0, 0.0, 1, 1)
    try:
        for call in (lambda: grs.grs_tensors_norm_sq(h, 8, 0, 1, 16, 8, 0),
                     lambda: grs.grs_tensors_adamw_step(h, hp, None, 8, 0, 16, 16, 16, None, 0),
                     lambda: grs.grs_tensors_adamw8_step(h, hp, 1, None, 8, 0, 16, 16, 4, 16, 4, None, 0),
                     lambda: grs.grs_tensors_pack8(h, 16, 16, 16, 4, 16, 4, 0),
                     lambda: grs.grs_tensors_unpack8(h, 16, 4, 16, 4, 16, 16, 0)):
            with pytest.raises(grs.GrsError) as e:
                call()
            assert e.value.status == grs.GRS_ERR_NO_DEVICE
        assert grs.grs_tensors_check_device_errors(h, 0) == grs.GRS_ERR_NO_DEVICE
        with pytest.raises(grs.GrsError) as e:
            grs.grs_tensors_offset(h, 1)
        assert e.value.status == grs.GRS_ERR_INVALID_ARG
    finally:
        grs.grs_tensors_destroy(h)


def test_null_handles_are_refused(grs):
    for call in (lambda: grs.grs_tensors_query(None), lambda: grs.grs_tensors_offset(None, 0),
                 lambda: grs.grs_tensors_norm_sq(None, 8, 0, 1, 16, 8, 0)):
        with pytest.raises(grs.GrsError) as e:
            call()
        assert e.value.status == grs.GRS_ERR_INVALID_ARG
    grs.grs_tensors_destroy(None)
