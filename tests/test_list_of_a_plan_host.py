"""A plan's arrays as a list of one tensor: how long the state arrays are."""
import os
import re

import pytest

import workloads

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def grs():
    from gradient_reduction_sharded_gb300 import _build
    _build.build()
    from gradient_reduction_sharded_gb300 import grs as g
    return g


def test_the_lists_states_are_longer_than_the_plans(grs):
    longer = []
    for i in range(3):
        w = workloads.get(i)
        plan = grs.grs_plan_create(w.numels, w.owners, w.world, w.tp, w.dp_replicate, w.dp_shard, w.bucket_bytes, flags=grs.GRS_PLAN_HOST_ONLY)
        n = grs.grs_plan_query(plan)["n_state_pad"]
        lst = grs.grs_tensors_create([n], grs.GRS_PLAN_HOST_ONLY)
        info = grs.grs_tensors_query(lst)
        assert info["n_state"] == -(-n // 256) * 256
        longer.append(info["n_state"] - n)
        grs.grs_tensors_destroy(lst)
        grs.grs_plan_destroy(plan)
    assert max(longer) > 0  # so what the header says of them matters
    with open(os.path.join(ROOT, "include", "grs.h")) as f:
        header = re.sub(r"[\s*]+", " ", f.read())
    assert "have the list's n_state elements" in header


def test_the_example_allocates_them(grs):
    with open(os.path.join(ROOT, "examples", "moe_block_step.py")) as f:
        assert "torch.zeros(ns - n, device=dev)" in f.read()
