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


# (requests, heads of keys, of values, Dk, Dv, tokens): one, two and four slices of 16 rows a block of several chunks, of one
# short one, and whole heads
WALKS = [(3, 2, 4, 128, 128, 200), (6, 2, 4, 128, 128, 200), (24, 2, 4, 64, 64, 130), (3, 2, 4, 128, 128, 32),
         (12, 2, 4, 128, 128, 32), (40, 2, 4, 128, 128, 32), (40, 2, 4, 128, 128, 140)]


@pytest.mark.parametrize("R,Hk,Hv,Dk,Dv,n", WALKS)
def test_a_state_is_left_or_right_after_a_timeout(R, Hk, Hv, Dk, Dv, n):
    """In place, with waits that run out at once: what a block of the walk did not finish it does not store, so each 16 rows of
    a state are either what they were or what they should become."""
    dd = ms.DeltaDims(Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, n_slots=R)
    s = make(dd, R, n, 61)
    start, ws = s["state"].clone(), ms.delta_workspace(dd, R, n)
    right = torch.empty_like(start)
    _, word = call(dd, R, s, ws=ws, state_out=right)
    assert word == ms.OK
    for _ in range(5):
        s["state"].copy_(start)
        try:
            ms.set_wait_timeout_ns(0)
            _, word = call(dd, R, s, ws=ws, state_out=s["state"])
        finally:
            ms.set_wait_timeout_ns(2_000_000_000)
        assert word == ms.ETIMEOUT
        cut = lambda t: t.view(R, Hv, Dv // 16, 16 * Dk)  # noqa: E731
        left, done = ((cut(s["state"]) == cut(x)).all(-1) for x in (start, right))
        assert (left | done).all(), int((~(left | done)).sum())
    s["state"].copy_(start)
    _, word = call(dd, R, s, ws=ws, state_out=s["state"])
    assert word == ms.OK and torch.equal(s["state"], right)
