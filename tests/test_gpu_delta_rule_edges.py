"""block_delta_rule at its edges."""
import pytest
import torch

import moe_expert_step_gb300 as ms
from tests.test_gpu_delta_rule import call, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,n", [(ms.F32, 6), (ms.BF16, 6), (ms.BF16, 24), (ms.BF16, 90)])
@pytest.mark.parametrize("k_exp,q_exp", [(-70, 0), (-80, 0), (-110, 0), (0, -80), (0, -110), (-60, -60)])
def test_tiny_keys_and_queries(dtype, n, k_exp, q_exp):
    """Keys and queries far below sqrt(qk_eps) are divided by that, not by zero or infinity; new requests, so that what they
    write and read is all there is."""
    dd = ms.DeltaDims(Hk=1, Hv=2, Dk=64, Dv=64, n_slots=2, dtype=dtype)
    s = make(dd, 2, n, 300 + n)
    s["k"], s["q"] = s["k"] * 2.0 ** k_exp, s["q"] * 2.0 ** q_exp
    fresh, to = torch.ones(2, dtype=torch.uint8, device="cuda"), torch.empty_like(s["state"])
    out, word = call(dd, 2, s, state_out=to, fresh=fresh)
    assert word == ms.OK
    check(dd, 2, s, out, to, fresh=fresh)
