"""block_attention in the orders of segments, row tiles and windows that its division of the work can
bring, against the float64 oracle with the bounds of test_gpu_attention.py."""
import pytest
import torch

import moe_expert_step_gb300 as ms
from tests.test_gpu_attention import Setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n_q", [4, 8, 16])
@pytest.mark.parametrize("dtype", [ms.BF16, ms.FP8])
def test_segments_that_one_stream_has_no_tile_of(dtype, n_q, D):
    """Row tiles of 32, 64 and 128; every CTA goes through three segments of one key tile, which the
    second stream only passes."""
    s = Setup(dtype, [1 + (7 * r) % 12 for r in range(57)], n_q, Hkv=8, G=8, D=D, page=16, seed=21)
    out, ls = s.run()
    s.check(out, ls)
    for _ in range(20):
        o2, l2 = s.run()
        assert torch.equal(o2, out) and torch.equal(l2, ls)
