"""block_delta_rule at its edges."""
import numpy as np
import pytest
import torch

import moe_expert_step_gb300 as ms
from oracle import token_mixer as om
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


@pytest.mark.parametrize("Hk,Hv,Dk,Dv", [(1, 2, 64, 64), (2, 2, 128, 128), (1, 3, 128, 64), (2, 4, 64, 128)])
@pytest.mark.parametrize("R,n", [(1, 1), (3, 1), (2, 2), (5, 5), (1, 16), (2, 17), (3, 23)])
def test_tokens_in_bf16_are_held_to_the_bound_of_fp32(Hk, Hv, Dk, Dv, R, n):
    """Up to 23 tokens a call bf16 goes token by token in fp32: 40 units of 2^-24 a token and the output's own rounding, without
    the f16 numbers of the chunked form."""
    dd = ms.DeltaDims(Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, n_slots=R)
    assert ms.delta_workspace_size(dd, R, n) == 512  # (no tiles: not in chunks)
    s = make(dd, R, n, 40 * n + R, extra=8)
    to = torch.empty_like(s["state"])
    out, word = call(dd, R, s, state_out=to, scale=Dk ** -0.5)
    assert word == ms.OK
    check(dd, R, s, out, to, scale=Dk ** -0.5, chunks=False)


@pytest.mark.parametrize("R,Hk,Hv,Dk,Dv,n", [(1, 1, 2, 64, 64, 4001), (1, 1, 1, 128, 128, 2500), (40, 1, 2, 64, 128, 900)])
def test_long_calls(R, Hk, Hv, Dk, Dv, n):
    """Thousands of tokens with decays and rates as they come, against the recurrence token by token.  (The long ones of a
    ragged batch; many heads of 128 values are walked a head a block.)"""
    dd = ms.DeltaDims(Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, n_slots=R)
    s = make(dd, R, n, 900 + R, decay=0.5)
    length = torch.tensor([n - (211 * r) % n for r in range(R)], dtype=torch.int32, device="cuda")
    to = torch.empty_like(s["state"])
    out, word = call(dd, R, s, state_out=to, length=length, scale=Dk ** -0.5)
    assert word == ms.OK
    one = ms.DeltaDims(Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, n_slots=1)
    for r in range(0, R, 7):
        part = {k: (v[r:r + 1] if k == "state" else v[r * n:(r + 1) * n]) for k, v in s.items()}
        check(one, 1, part, out[r * n:(r + 1) * n], to[r:r + 1], length=length[r:r + 1], scale=Dk ** -0.5)


@pytest.mark.parametrize("R,Hk,Hv,Dk,Dv,n", [(3, 2, 4, 128, 128, 200), (40, 2, 4, 128, 128, 200), (3, 2, 4, 64, 64, 32)])
@pytest.mark.parametrize("what", ["q", "k", "v", "g", "beta"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_what_a_non_finite_value_reaches(R, Hk, Hv, Dk, Dv, n, what, value):
    """In chunks it may reach its head's outputs from the beginning of its chunk of 64 tokens on and its head's state; nothing
    before that, no other head, no other request."""
    if what == "g" and value < 0:
        pytest.skip("a history that is dropped is finite")
    dd = ms.DeltaDims(Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, n_slots=R)
    s = make(dd, R, n, 17)
    clean_to, to = torch.empty_like(s["state"]), torch.empty_like(s["state"])
    clean, word = call(dd, R, s, state_out=clean_to)
    assert word == ms.OK
    r, t, head = R // 2, min(n - 1, 70), 1
    bad = dict(s, **{what: s[what].clone()})
    bad[what].view(R, n, *s[what].shape[1:])[r, t, head].view(-1)[0] = value
    out, word = call(dd, R, bad, state_out=to)
    assert word == ms.OK
    heads = [head] if what in ("v", "g", "beta") else [2 * head, 2 * head + 1]
    same = (out == clean).view(R, n, Hv, Dv).all(-1)
    reached = torch.zeros((R, n, Hv), dtype=torch.bool, device="cuda")
    reached[r, t // 64 * 64:, heads] = True
    assert same[~reached].all()
    states = (to == clean_to).flatten(2).all(-1)
    reached = torch.zeros((R, Hv), dtype=torch.bool, device="cuda")
    if what != "q":
        reached[r, heads] = True
    assert states[~reached].all()
    for h in heads:  # and its own token's output shows it
        assert not out.view(R, n, Hv, Dv)[r, t, h].isfinite().all()


@pytest.mark.parametrize("n,start", [(32, 0), (32, 9), (64, 0), (64, 25), (150, 70)])
def test_a_rule_that_grows_within_its_limit(n, start):
    """14 tokens of one key with beta |k|^2 = 3: each doubles what the one before wrote, 2^14 in all, just below the limit of
    the chunked form; the others have beta = 0.  Operands are pairs of f16 numbers, off by 2^-22, and a row of the inverse
    has entries of alternating signs that add up to 2^14 with the last: at most three roundings of 28 products of the size of
    the result, 2^-22 * 3 * 28 < 2^-15, and 2^-14 of the state's norm is allowed."""
    dd = ms.DeltaDims(Hk=1, Hv=1, Dk=64, Dv=64, n_slots=1)
    s = make(dd, 1, n, 5)
    s["k"] = torch.full_like(s["k"], 0.25)  # |k|^2 = 4
    s["beta"] = torch.zeros_like(s["beta"])
    s["beta"][start:start + 14] = 0.75
    s["g"] = torch.zeros_like(s["g"])
    to = torch.empty_like(s["state"])
    out, word = call(dd, 1, s, state_out=to, qk_eps=0.0)
    assert word == ms.OK
    x = {k: v.double().cpu().numpy() for k, v in s.items()}
    want, S, _ = om.delta_rule(x["q"], x["k"], x["v"], x["g"], x["beta"], x["state"][0], 1.0, 0.0)
    assert np.linalg.norm(S) > 2.0 ** 13 * np.linalg.norm(x["state"][0]) / 16
    off = np.linalg.norm(to[0].double().cpu().numpy() - S) / np.linalg.norm(S)
    assert off <= 2.0 ** -14, off
    off = np.linalg.norm(out.double().cpu().numpy() - want) / np.linalg.norm(want)
    assert off <= 2.0 ** -8 + 2.0 ** -11, off


@pytest.mark.parametrize("R,Hk,Hv,Dk,Dv,n", WALKS)
@pytest.mark.parametrize("larger", ["history", "values"])
def test_a_history_that_is_dropped_within_a_chunk(R, Hk, Hv, Dk, Dv, n, larger):
    """A decay of -inf in the middle of 64 tokens (a sequence that ends, another one behind it), the first one's history or
    values 2^12 times the second one's.  In chunks a row's new values are off by 2^-22 of themselves or 2^-37 of the largest
    of 64 tokens, here 2^-25 of the second sequence's: within the bound of the norms."""
    dd = ms.DeltaDims(Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, n_slots=R)
    s = make(dd, R, n, 71)
    at = torch.tensor([(r * n + 11 + 5 * r % (n - 20)) for r in range(R)], device="cuda")
    s["g"][at] = float("-inf")
    if larger == "history":
        s["state"] *= 2.0 ** 12
    else:
        before = torch.arange(R * n, device="cuda") < at.repeat_interleave(n)
        s["v"] = torch.where(before[:, None, None], s["v"] * 2.0 ** 12, s["v"])
    to = torch.empty_like(s["state"])
    out, word = call(dd, R, s, state_out=to, scale=Dk ** -0.5)
    assert word == ms.OK
    check(dd, R, s, out, to, scale=Dk ** -0.5)


def test_whole_heads_and_attention_follow_each_other():
    """Both take tensor memory, and each may start while the other's blocks still run: many in a row give what each gives alone."""
    R, n, T = 40, 140, 32
    dd = ms.DeltaDims(Hk=2, Hv=4, Dk=128, Dv=128, n_slots=R)
    s = make(dd, R, n, 91)
    kd = ms.KvDims(Hq=16, Hkv=2, D=128, page=64, n_pages=R * 8, max_pages=8)
    z = lambda *shape: torch.randn(shape, device="cuda").bfloat16()  # noqa: E731
    table = torch.arange(R * 8, dtype=torch.int32, device="cuda").view(R, 8)
    cache, q = ms.kv_cache(z(R * 8, 2, 64, 128), z(R * 8, 2, 64, 128), table), z(R * T, 16, 128)
    seen = torch.randint(T, 513, (R,), device="cuda").to(torch.int32)
    kv_ws, ws = ms.kv_workspace(kd, R, T), ms.delta_workspace(dd, R, n)
    want, word = call(dd, R, s, ws=ws)
    assert word == ms.OK
    att = torch.empty_like(q)
    ms.block_attention(kd, R, q, seen, cache, att, kv_ws, 128 ** -0.5)
    torch.cuda.synchronize()
    outs = [(torch.zeros_like(want), torch.zeros_like(att)) for _ in range(30)]
    for o, a in outs:
        ms.block_delta_rule(dd, R, s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], o, ws, qk_eps=1e-6)
        ms.block_attention(kd, R, q, seen, cache, a, kv_ws, 128 ** -0.5)
    torch.cuda.synchronize()
    assert ms.read_device_error(ws) == ms.OK and ms.read_device_error(kv_ws) == ms.OK
    assert all(torch.equal(o, want) and torch.equal(a, att) for o, a in outs)
