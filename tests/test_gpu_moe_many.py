"""Tokens to experts and back where the launch changes shape: many tokens, and
every number of rows in flight.  The checks are those of ordinary sizes."""
import pytest

import test_gpu_moe
from test_gpu_moe import grs  # noqa: F401

pytestmark = pytest.mark.gpu

# 2432 tokens are many; k of 1 .. 9 takes each kernel and its loop; the widths one warp, several, and a part of the last
SHAPES = [(2431, 4, 1024), (2432, 1, 512), (2500, 3, 2048), (2433, 5, 4096), (2440, 6, 1536), (2432, 2, 264), (3000, 7, 776),
          (2432, 9, 64), (2600, 1, 4104), (2500, 2, 2051), (2432, 8, 8200)]


@pytest.mark.parametrize("tokens,k,d", SHAPES)
@pytest.mark.parametrize("act,begin,end,shift", [("bf16", 0, 6, 0), ("fp32", 0, 6, 0), ("bf16", 2, 5, 0)])
def test_vectors_of_many_tokens(grs, tokens, k, d, act, begin, end, shift):  # noqa: F811
    test_gpu_moe.test_vectors_there_and_back(grs, tokens, k, d, act, begin, end, shift)
