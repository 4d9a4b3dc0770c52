"""block_attention over FP8 caches with keys and queries of any size that the cache's exponents and bf16
can express, against the float64 oracle with the bounds of test_gpu_attention.py: powers of two change
neither the relative errors nor the weights, as long as the scale takes them back."""
import pytest
import torch

import moe_expert_step_gb300 as ms
from tests.test_gpu_attention import Setup

pytestmark = pytest.mark.gpu


def scaled(keys, queries, n_q, D, seed=30):
    """A setup whose keys are 2^keys and queries 2^queries times as large, its scale as much smaller."""
    s = Setup(ms.FP8, [300, 33], n_q, 1, 2, D, 32, seed=seed)
    ek, tab = s.cache._tensors[3], s.table.cpu().numpy()
    for r, L in enumerate(s.lengths):
        for j in range(L):
            i = (int(tab[r, j // 32]), 0, j % 32)
            ek[i] = int(ek[i]) + keys
        s.k[r] = s.k[r].astype("float64") * 2.0 ** keys
    s.q = (s.q.double() * 2.0 ** queries).bfloat16()
    s.scale *= 2.0 ** -(keys + queries)
    return s


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n_q", [3, 20, 50, 80])
@pytest.mark.parametrize("keys,queries", [(120, -84), (112, -60), (-93, 100), (-80, 118), (60, 30), (-93, -20)])
def test_large_and_small_keys(keys, queries, n_q, D):
    """Row tiles of 32, 64, 128 and 256; exponents from -100 to 119, queries from 2^-84 to 2^120."""
    s = scaled(keys, queries, n_q, D)
    s.check(*s.run())


@pytest.mark.parametrize("n_q", [3, 20, 50, 80])
def test_large_queries_beside_ordinary_ones(n_q):
    """Rows of one tile whose powers of two lie 80 apart."""
    s = scaled(-60, 0, n_q, 128)
    s.scale *= 2.0 ** -40
    f = torch.tensor([2.0 ** (40 * (i % 3)) for i in range(s.q.shape[0])], dtype=torch.float64, device="cuda")
    s.q = (s.q.double() * f[:, None, None]).bfloat16()
    s.check(*s.run())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n_q", [3, 20, 50, 80])
@pytest.mark.parametrize("keys,queries", [(96, -96), (112, -112), (118, -115)])
def test_tiny_queries(keys, queries, n_q, D):
    """Queries down to 2^-115 keep their bits."""
    s = scaled(keys, queries, n_q, D, seed=31)
    s.check(*s.run())
