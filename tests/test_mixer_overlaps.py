"""Outputs of block_delta_rule in place of its inputs are refused (CPU, at the C entry): other blocks still read them."""
import pytest

import moe_expert_step_gb300 as ms

PLACE = {name: (i + 1) << 20 for i, name in enumerate(("q", "k", "v", "g", "beta", "state", "out", "ws"))}


@pytest.mark.parametrize("n,dtype", [(1, ms.BF16), (4, ms.F32), (32, ms.BF16), (200, ms.BF16)])
@pytest.mark.parametrize("other", ["q", "k", "state", "state_out"])
def test_out_in_the_place_of_an_input(n, dtype, other):
    if not ms.os.path.exists(ms.library_path()):
        ms.build()
    dd = ms.DeltaDims(Hk=2, Hv=2, Dk=64, Dv=64, n_slots=2, dtype=dtype)
    p = dict(PLACE, state_out=9 << 20)
    p["out"] = p[other]
    rc = ms.lib().block_delta_rule(dd._c, 2, n, p["q"], 128, p["k"], 128, p["v"], 128, p["g"], p["beta"], None, None, None,
                                   p["state"], p["state_out"], 1.0, 0.0, p["out"], p["ws"], 1 << 40, None)
    assert rc == ms.EINVAL
