"""block_delta_rule against the float64 recurrence.

Bound.  With |k| <= 1 and 0 <= beta <= 1 a token maps a row of the state by a contraction, so errors add up over
the tokens and never grow.  Let M be the largest norm of the row plus the largest |v| of it, u = 2^-24.  A token's own
error, token by token in fp32: the product with k (sums of 16 and 3 steps) 20 u, the normalised key 6 u, the decay
and the rest of the formula 8 u, of M each: 34 u M, 40 u M are allowed.  In chunks of 64 tokens the operands are pairs
of f16 numbers (2^-22 = 4 u of a value each, two factors to a product, products of 64 or 128 terms 40 u) and a token's
error enters the 63 others of its chunk through entries of the inverse that are at most 1: 64 * 60 u M.  Both
bounds are for every element in the worst case; errors of independent signs give the square root of their number, and
of the whole state's norm 2^-17 is allowed for that (measured values are below 2^-20).  Outputs: the same bound with
|q| <= 1, times the scale, and the rounding to their type; in chunks the output products take one f16 number (2^-12 of each
factor: 2^-11 M in all)."""
import numpy as np
import pytest
import torch

import moe_expert_step_gb300 as ms
from oracle import token_mixer as om

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def make(dd, R, n, seed, extra=0, decay=2.0, like=0.5):
    """Projected rows (wider than needed by `extra`), gates, a pool of states."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    act = torch.float32 if dd.dtype == ms.F32 else torch.bfloat16
    T, wk, wv = R * n, dd.Hk * dd.Dk, dd.Hv * dd.Dv
    x = torch.randn((T, 2 * wk + wv + extra), generator=g, device="cuda") + like * torch.randn(
        2 * wk + wv + extra, generator=g, device="cuda")
    x = x.to(act)
    s = dict(q=x[:, :wk].unflatten(1, (dd.Hk, dd.Dk)), k=x[:, wk:2 * wk].unflatten(1, (dd.Hk, dd.Dk)),
             v=x[:, 2 * wk:2 * wk + wv].unflatten(1, (dd.Hv, dd.Dv)))
    rate = torch.exp(torch.empty(dd.Hv, device="cuda").uniform_(-9.0, float(np.log(decay)), generator=g))
    s["g"] = -rate * torch.exp(0.5 * torch.randn((T, dd.Hv), generator=g, device="cuda"))
    s["beta"] = torch.sigmoid(1.5 * torch.randn((T, dd.Hv), generator=g, device="cuda"))
    s["state"] = 0.3 * torch.randn((dd.n_slots, dd.Hv, dd.Dv, dd.Dk), generator=g, device="cuda")
    return s


def call(dd, R, s, **kw):
    T = s["q"].shape[0]
    out = torch.full((T, dd.Hv, dd.Dv), 5.0, device="cuda", dtype=s["q"].dtype)
    ws = kw.pop("ws", None)
    ws = ms.delta_workspace(dd, R, T // R) if ws is None else ws
    kw.setdefault("qk_eps", 1e-6)
    ms.block_delta_rule(dd, R, s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], out, ws, **kw)
    torch.cuda.synchronize()
    return out, ms.read_device_error(ws)


def check(dd, R, s, out, state_out, slot=None, length=None, fresh=None, scale=1.0, qk_eps=1e-6, chunks=None):
    T = s["q"].shape[0]
    n = T // R
    np64 = {k: v.double().cpu().numpy() for k, v in s.items()}
    got, pool = out.double().cpu().numpy().reshape(R, n, dd.Hv, dd.Dv), None
    if state_out is not None:
        pool = state_out.double().cpu().numpy()
    tokens = 64 * 60 * U if (dd.dtype == ms.BF16 if chunks is None else chunks) else 40 * U
    inner = 2.0 ** -11 if tokens > 1000 * U else 0.0
    for r in range(R):
        i, m = (r if slot is None else int(slot[r])), (n if length is None else int(length[r]))
        rows = slice(r * n, r * n + m)
        assert (got[r, m:] == 5.0).all() if i >= 0 else (got[r] == 5.0).all()
        if i < 0:
            continue
        S0 = np64["state"][i] * (0.0 if fresh is not None and fresh[r] else 1.0)
        want, S, most = om.delta_rule(np64["q"][rows], np64["k"][rows], np64["v"][rows], np64["g"][rows],
                                      np64["beta"][rows], S0, scale, qk_eps)
        err = tokens * max(m, 1) * most
        tol = scale * (err + inner * most)[None] + (2.0 ** -8 if dd.dtype == ms.BF16 else U) * np.abs(want)
        assert (np.abs(got[r, :m] - want) <= tol + 1e-30).all(), float((np.abs(got[r, :m] - want) / tol).max())
        if m:
            off = np.linalg.norm(got[r, :m] - want) / np.linalg.norm(want)
            assert off <= (2.0 ** -8 if dd.dtype == ms.BF16 else 2.0 ** -17), off
        if pool is not None:
            e = np.sqrt(((pool[i] - S) ** 2).sum(-1))
            assert (e <= err + 2.0 ** -23 * most).all(), float((e / err).max())
            # (a state that has decayed below 2^-126, the smallest normal number of fp32, may be zero: off by 2^-126 an element)
            assert np.linalg.norm(pool[i] - S) <= 2.0 ** -17 * np.linalg.norm(S) + 2.0 ** -126 * np.sqrt(S.size)


SHAPES = [(1, 2, 64, 64), (2, 2, 128, 128), (1, 3, 128, 64), (2, 4, 64, 128)]


@pytest.mark.parametrize("dtype", [ms.F32, ms.BF16])
@pytest.mark.parametrize("Hk,Hv,Dk,Dv", SHAPES)
@pytest.mark.parametrize("R,n", [(1, 1), (3, 1), (2, 2), (1, 16), (2, 17), (3, 33), (1, 100)])
def test_short(dtype, Hk, Hv, Dk, Dv, R, n):
    dd = ms.DeltaDims(Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, n_slots=R + 2, dtype=dtype)
    s = make(dd, R, n, 100 * n + R, extra=8)
    keep = s["state"].clone()
    slot = torch.randperm(R + 2, device="cuda")[:R].to(torch.int32)
    to = torch.full_like(s["state"], 3.0)
    out, word = call(dd, R, s, state_out=to, slot=slot, scale=Dk ** -0.5)
    assert word == ms.OK and torch.equal(s["state"], keep)
    check(dd, R, s, out, to, slot=slot, scale=Dk ** -0.5)
    others = [i for i in range(R + 2) if i not in slot.tolist()]
    assert (to[others] == 3.0).all()


@pytest.mark.parametrize("dtype", [ms.F32, ms.BF16])
@pytest.mark.parametrize("n", [5, 150])
def test_lengths_slots_fresh(dtype, n):
    """Ragged requests, an idle one, one without tokens, one that begins from nothing in a slot of NaN; what stands
    behind a request's tokens may be anything; a history that is only read stays."""
    dd = ms.DeltaDims(Hk=1, Hv=2, Dk=64, Dv=64, n_slots=7, dtype=dtype)
    R = 6
    s = make(dd, R, n, 8)
    length = torch.tensor([n, 0, 1, n // 2, n - 1, n], dtype=torch.int32, device="cuda")
    slot = torch.tensor([6, 3, 0, -1, 5, 1], dtype=torch.int32, device="cuda")
    fresh = torch.tensor([0, 0, 1, 0, 1, 0], dtype=torch.uint8, device="cuda")
    s["state"][0] = float("nan")
    s["state"][2] = float("nan")
    for r in range(R):
        for x in ("q", "k", "v", "g", "beta"):
            s[x][r * n + int(length[r]):(r + 1) * n] = float("nan")
    before = s["state"].clone()
    out, word = call(dd, R, s, slot=slot, length=length, fresh=fresh)
    assert word == ms.OK and torch.equal(s["state"].nan_to_num(9.0), before.nan_to_num(9.0))
    clean = {k: v.nan_to_num(0.0) for k, v in s.items()}
    check(dd, R, clean, out, None, slot=slot, length=length, fresh=fresh)
    out2, word = call(dd, R, s, slot=slot, length=length, fresh=fresh, state_out=s["state"])
    assert word == ms.OK and torch.equal(out, out2)
    check(dd, R, clean, out2, s["state"], slot=slot, length=length, fresh=fresh)
    assert torch.equal(s["state"][3], before[3]) and torch.isnan(s["state"][2]).all()
    assert torch.equal(s["state"][4], before[4])


@pytest.mark.parametrize("dtype", [ms.F32, ms.BF16])
@pytest.mark.parametrize("what,value", [("length", -1), ("length", 71), ("slot", 3), ("slot", 2 ** 31 - 1)])
@pytest.mark.parametrize("n", [4, 70])
def test_bad_values_are_recorded(dtype, what, value, n):
    dd = ms.DeltaDims(Hk=1, Hv=1, Dk=64, Dv=64, n_slots=3, dtype=dtype)
    if what == "length" and value > 0:
        value = n + 1
    s = make(dd, 3, n, 4)
    kw = dict(length=[n, n, n], slot=[0, 1, 2])
    kw[what][1] = value
    t = {k: torch.tensor(v, dtype=torch.int32, device="cuda") for k, v in kw.items()}
    to = torch.full_like(s["state"], 3.0)
    out, word = call(dd, 3, s, state_out=to, **t)
    assert word == ms.EDEVINPUT
    assert (out[n:2 * n] == 5.0).all() and (to[1] == 3.0).all()
    kw["slot"][1] = -1  # skipped: as if it were not there
    if what == "length":
        kw["length"][1] = n
    check(dd, 3, s, out, to, length=kw["length"], slot=kw["slot"])


@pytest.mark.parametrize("dtype", [ms.F32, ms.BF16])
@pytest.mark.parametrize("n", [3, 65])
def test_decays(dtype, n):
    """Histories that are dropped (-inf), hardly decay, or decay by more than fp32 holds, next to one another."""
    dd = ms.DeltaDims(Hk=1, Hv=3, Dk=64, Dv=64, n_slots=1, dtype=dtype)
    s = make(dd, 1, n, 14)
    s["g"][:, 0] = torch.where(torch.arange(n, device="cuda") % 2 == 1, float("-inf"), -1e-3)
    s["g"][:, 1] = torch.where(torch.arange(n, device="cuda") % 3 == 1, -90.0, -1e-6)
    s["g"][:, 2] = torch.where(torch.arange(n, device="cuda") % 5 == 1, -3e38, 0.0)
    to = torch.empty_like(s["state"])
    out, word = call(dd, 1, s, state_out=to)
    assert word == ms.OK
    check(dd, 1, s, out, to)


@pytest.mark.parametrize("dtype", [ms.F32, ms.BF16])
@pytest.mark.parametrize("n", [4, 96])
def test_without_normalisation(dtype, n):
    """Keys of length 1/2 as they are, and beta 0 or 1."""
    dd = ms.DeltaDims(Hk=2, Hv=2, Dk=64, Dv=128, n_slots=1, dtype=dtype)
    s = make(dd, 1, n, 15)
    act = s["k"].dtype
    s["k"], s["q"] = ((0.5 * x.float() / x.float().norm(dim=-1, keepdim=True)).to(act) for x in (s["k"], s["q"]))
    s["beta"] = (torch.rand_like(s["beta"]) < 0.5).float()
    to = torch.empty_like(s["state"])
    out, word = call(dd, 1, s, state_out=to, qk_eps=0.0)
    assert word == ms.OK
    check(dd, 1, s, out, to, qk_eps=0.0)


@pytest.mark.parametrize("n", [1, 32, 200])
def test_same_call_same_bits_captured_and_on_a_stream(n):
    dd = ms.DeltaDims(Hk=2, Hv=4, Dk=128, Dv=128, n_slots=5)
    s = make(dd, 5, n, 30)
    to = torch.empty_like(s["state"])
    a, _ = call(dd, 5, s, state_out=to)
    first = to.clone()
    to.zero_()
    stream, ws = torch.cuda.Stream(), ms.delta_workspace(dd, 5, n)
    torch.cuda.synchronize()
    b, _ = call(dd, 5, s, state_out=to, ws=ws, stream=stream)
    assert torch.equal(a, b) and torch.equal(first, to)
    out = torch.zeros_like(a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ms.block_delta_rule(dd, 5, s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], out, ws, state_out=to,
                            qk_eps=1e-6)
    for _ in range(3):
        out.zero_(), to.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, out) and torch.equal(first, to)


@pytest.mark.parametrize("dtype", [ms.F32, ms.BF16])
def test_pieces_of_a_sequence(dtype):
    """A sequence passed in pieces, in place, ends where the whole one does."""
    dd = ms.DeltaDims(Hk=1, Hv=2, Dk=128, Dv=64, n_slots=1, dtype=dtype)
    n = 260
    s = make(dd, 1, n, 44)
    start = s["state"].clone()
    at = 0
    outs = []
    for m in (1, 64, 2, 128, 65):
        part = {k: (v if k == "state" else v[at:at + m]) for k, v in s.items()}
        out, word = call(dd, 1, part, state_out=s["state"], scale=0.1)
        assert word == ms.OK
        outs.append(out)
        at += m
    assert at == n
    end, s["state"] = s["state"], start
    check(dd, 1, s, torch.cat(outs), end, scale=0.1)


def test_wait_timeout_is_reported_and_recovered():
    """Waits that run out end the walk with an error; the next call is right."""
    dd = ms.DeltaDims(Hk=2, Hv=4, Dk=128, Dv=128, n_slots=3)
    s = make(dd, 3, 200, 61)
    ws, to = ms.delta_workspace(dd, 3, 200), torch.empty_like(s["state"])
    good, word = call(dd, 3, s, ws=ws, state_out=to)
    first = to.clone()
    assert word == ms.OK
    try:
        ms.set_wait_timeout_ns(0)
        _, word = call(dd, 3, s, ws=ws, state_out=to)
        assert word == ms.ETIMEOUT
    finally:
        ms.set_wait_timeout_ns(2_000_000_000)
    again, word = call(dd, 3, s, ws=ws, state_out=to)
    assert word == ms.OK and torch.equal(good, again) and torch.equal(first, to)


@pytest.mark.parametrize("R,Hk,Hv", [(1, 1, 2), (5, 2, 6), (40, 4, 4)])
@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
def test_longer(R, Hk, Hv, Dk, Dv):
    """Several chunks, ragged, few and many slices of the states a multiprocessor, groups of one to three value heads.
    (Many heads of 128 values are walked in another way than few, so 40 requests of them go to the oracle one and all.)"""
    dd = ms.DeltaDims(Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, n_slots=R)
    n = 330 if R < 40 else 140
    s = make(dd, R, n, 70 + R)
    length = torch.tensor([n - (37 * r) % n for r in range(R)], dtype=torch.int32, device="cuda")
    to = torch.full_like(s["state"], 3.0)
    out, word = call(dd, R, s, state_out=to, length=length, scale=Dk ** -0.5)
    assert word == ms.OK
    if R == 40 and Dv == 64:  # the oracle on a few of them, the others against calls of their own
        for r in (0, 17, 39):
            part = {k: (v[r:r + 1] if k == "state" else v[r * n:(r + 1) * n]) for k, v in s.items()}
            check(ms.DeltaDims(Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, n_slots=1), 1, part, out[r * n:(r + 1) * n], to[r:r + 1],
                  length=length[r:r + 1], scale=Dk ** -0.5)
        for r in range(R):
            one = ms.DeltaDims(Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, n_slots=1)
            part = {k: (v[r:r + 1] if k == "state" else v[r * n:(r + 1) * n]) for k, v in s.items()}
            alone = torch.empty_like(part["state"])
            o, _ = call(one, 1, part, state_out=alone, length=length[r:r + 1], scale=Dk ** -0.5)
            assert torch.equal(o, out[r * n:(r + 1) * n]) and torch.equal(alone[0], to[r])
    else:
        check(dd, R, s, out, to, length=length, scale=Dk ** -0.5)


@pytest.mark.parametrize("n", [6, 100])
def test_magnitudes(n):
    """Values, states, queries and keys of very different sizes: powers of two of each change nothing but the result's."""
    dd = ms.DeltaDims(Hk=1, Hv=2, Dk=64, Dv=64, n_slots=1)
    s = make(dd, 1, n, 81)
    to = torch.empty_like(s["state"])
    out, _ = call(dd, 1, s, state_out=to, qk_eps=1e-30)
    for v, k, q in ((2.0 ** 60, 1.0, 1.0), (2.0 ** -60, 1.0, 1.0), (1.0, 2.0 ** 30, 2.0 ** -30), (1.0, 2.0 ** -30, 2.0 ** 40)):
        t = dict(s, v=s["v"] * v, state=s["state"] * v, k=s["k"] * k, q=s["q"] * q)
        to2 = torch.empty_like(to)
        out2, word = call(dd, 1, t, state_out=to2, qk_eps=1e-30)
        assert word == ms.OK
        assert (out2.double() / v - out.double()).abs().max() <= 2.0 ** -8 * out.double().abs().max()
        assert ((to2.double() / v - to.double()).norm() / to.double().norm()) <= 2.0 ** -17


@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("R,Hk,Hv", [(3, 1, 1), (24, 1, 3), (60, 2, 2)])
@pytest.mark.parametrize("n", [24, 31, 32])
def test_blocks(n, R, Hk, Hv, Dk, Dv):
    """One short chunk; few and many slices of the states a multiprocessor; ragged, idle and new requests, NaN behind a
    request's tokens; the history read only, written elsewhere, in place."""
    dd = ms.DeltaDims(Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, n_slots=R + 1)
    s = make(dd, R, n, 900 + n + R, extra=16)
    length = torch.tensor([[n, 0, 1, 15, 16, 17, n - 1, n // 2][r % 8] for r in range(R)], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(n)
    slot = torch.randperm(R + 1, generator=g)[:R].to(torch.int32).cuda()
    slot[R // 2] = -1
    fresh = (torch.rand(R, generator=g) < 0.3).to(torch.uint8).cuda()
    for r in range(R):
        if fresh[r] and slot[r] >= 0:
            s["state"][int(slot[r])] = float("nan")
        for x in ("q", "k", "v", "g", "beta"):
            s[x][r * n + int(length[r]):(r + 1) * n] = float("nan")
    clean = {k: v.nan_to_num(0.0) for k, v in s.items()}
    kw = dict(slot=slot, length=length, fresh=fresh, scale=Dk ** -0.5)
    out, word = call(dd, R, s, **kw)
    assert word == ms.OK
    check(dd, R, clean, out, None, **kw)
    to = torch.full_like(s["state"], 3.0)
    out2, word = call(dd, R, s, state_out=to, **kw)
    assert word == ms.OK and torch.equal(out, out2)
    check(dd, R, clean, out, to, **kw)
    idle = [i for i in range(R + 1) if i not in slot.tolist()]
    assert (to[idle] == 3.0).all()
    out3, word = call(dd, R, s, state_out=s["state"], **kw)
    assert word == ms.OK and torch.equal(out, out3)
    used = [int(i) for i in slot if i >= 0]
    assert torch.equal(s["state"][used], to[used])


def test_blocks_are_their_sequence():
    """Blocks of 32 and of 24 in place end where one call over all of their tokens does; a block that is read only changes
    nothing; a wait that runs out is reported."""
    dd = ms.DeltaDims(Hk=1, Hv=2, Dk=128, Dv=128, n_slots=1)
    s = make(dd, 1, 120, 46)
    start, outs, at = s["state"].clone(), [], 0
    for m in (32, 24, 32, 32):
        part = {k: (v if k == "state" else v[at:at + m]) for k, v in s.items()}
        before = s["state"].clone()
        seen, word = call(dd, 1, part, scale=0.1)
        assert word == ms.OK and torch.equal(before, s["state"])
        out, word = call(dd, 1, part, state_out=s["state"], scale=0.1)
        assert word == ms.OK and torch.equal(seen, out)
        outs.append(out)
        at += m
    assert at == 120
    try:
        ms.set_wait_timeout_ns(0)
        _, word = call(dd, 1, {k: (v if k == "state" else v[:32]) for k, v in s.items()}, state_out=torch.empty_like(start))
        assert word == ms.ETIMEOUT
    finally:
        ms.set_wait_timeout_ns(2_000_000_000)
    end, s["state"] = s["state"], start
    check(dd, 1, s, torch.cat(outs), end, scale=0.1)


def many(R, Hk, Hv, Dk, n, seed, **kw):
    """More heads of 128 values than half the multiprocessors, more than one chunk: walked a head a block."""
    dd = ms.DeltaDims(Hk=Hk, Hv=Hv, Dk=Dk, Dv=128, n_slots=R + 2)
    assert 8 * R * Hv > 4 * torch.cuda.get_device_properties(0).multi_processor_count and n > 64
    return dd, make(dd, R, n, seed, **kw)


@pytest.mark.parametrize("Dk", [64, 128])
@pytest.mark.parametrize("Hk,Hv,n", [(1, 1, 65), (1, 1, 129), (1, 2, 200), (2, 6, 128)])
def test_many_heads(Dk, Hk, Hv, n):
    """Ragged, from no token to several chunks, idle requests, new ones in slots of NaN, NaN behind a request's tokens."""
    R = 84 // Hv
    dd, s = many(R, Hk, Hv, Dk, n, 500 + n + Dk, extra=8)
    length = torch.tensor([[n, 0, 1, 63, 64, 65, n - 1, n // 2][r % 8] for r in range(R)], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(n)
    slot = torch.randperm(R + 2, generator=g)[:R].to(torch.int32).cuda()
    slot[5] = -1
    fresh = (torch.rand(R, generator=g) < 0.3).to(torch.uint8).cuda()
    for r in range(R):
        if fresh[r] and slot[r] >= 0:
            s["state"][int(slot[r])] = float("nan")
        for x in ("q", "k", "v", "g", "beta"):
            s[x][r * n + int(length[r]):(r + 1) * n] = float("nan")
    clean = {k: v.nan_to_num(0.0) for k, v in s.items()}
    out, word = call(dd, R, s, slot=slot, length=length, fresh=fresh, scale=Dk ** -0.5)
    assert word == ms.OK
    check(dd, R, clean, out, None, slot=slot, length=length, fresh=fresh, scale=Dk ** -0.5)
    out2, word = call(dd, R, s, slot=slot, length=length, fresh=fresh, scale=Dk ** -0.5, state_out=s["state"])
    assert word == ms.OK and torch.equal(out, out2)
    check(dd, R, clean, out2, s["state"], slot=slot, length=length, fresh=fresh, scale=Dk ** -0.5)


def test_many_heads_decays_and_gates():
    """Histories dropped, kept, decaying by more than fp32 holds; gates of 0 and 1; states of zeros."""
    n, R = 150, 80
    dd, s = many(R, 1, 1, 128, n, 14)
    t = torch.arange(n, device="cuda")
    for r in range(R):
        rows = slice(r * n, (r + 1) * n)
        if r % 4 == 0:
            s["g"][rows, 0] = torch.where(t % 37 == 1, float("-inf"), -1e-3)
        elif r % 4 == 1:
            s["g"][rows, 0] = torch.where(t % 3 == 1, -90.0, -1e-6)
        elif r % 4 == 2:
            s["g"][rows, 0] = torch.where(t % 70 == 1, -3e38, 0.0)
        if r % 3 == 0:
            s["beta"][rows] = (torch.rand_like(s["beta"][rows]) < 0.5).float()
        if r % 5 == 0:
            s["state"][r] = 0.0
        if r % 7 == 0:
            s["beta"][rows][64:] = 0.0  # a chunk that adds nothing
    to = torch.empty_like(s["state"])
    out, word = call(dd, R, s, state_out=to)
    assert word == ms.OK
    check(dd, R, s, out, to)


def test_many_heads_magnitudes():
    """Values, states, queries and keys of very different sizes: powers of two of each change nothing but the result's; a
    history far above and far below what is added to it leaves the larger of both as it is alone."""
    n, R = 130, 80
    dd, s = many(R, 1, 1, 128, n, 81)
    to = torch.empty_like(s["state"])
    out, _ = call(dd, R, s, qk_eps=1e-30, state_out=to)
    used = slice(0, R)
    for v, k, q in ((2.0 ** 60, 1.0, 1.0), (2.0 ** -60, 1.0, 1.0), (1.0, 2.0 ** 30, 2.0 ** -30), (1.0, 2.0 ** -30, 2.0 ** 40)):
        t = dict(s, v=s["v"] * v, state=s["state"] * v, k=s["k"] * k, q=s["q"] * q)
        to2 = torch.empty_like(to)
        out2, word = call(dd, R, t, qk_eps=1e-30, state_out=to2)
        assert word == ms.OK
        assert (out2.double() / v - out.double()).abs().max() <= 2.0 ** -8 * out.double().abs().max()
        assert ((to2[used].double() / v - to[used].double()).norm() / to[used].double().norm()) <= 2.0 ** -17
    for sv, ss in ((2.0 ** 50, 2.0 ** -50), (2.0 ** -50, 2.0 ** 50)):
        t = dict(s, v=s["v"] * sv, state=s["state"] * ss)
        to2 = torch.empty_like(to)
        out2, word = call(dd, R, t, state_out=to2)
        assert word == ms.OK
        check(dd, R, t, out2, to2)


def test_many_heads_streams_graphs_and_timeouts():
    n, R = 140, 80
    dd, s = many(R, 1, 1, 128, n, 30)
    to = torch.empty_like(s["state"])
    a, word = call(dd, R, s, state_out=to)
    assert word == ms.OK
    first = to.clone()
    stream, ws = torch.cuda.Stream(), ms.delta_workspace(dd, R, n)
    torch.cuda.synchronize()
    b, _ = call(dd, R, s, state_out=to, ws=ws, stream=stream)
    assert torch.equal(a, b) and torch.equal(first, to)
    try:
        ms.set_wait_timeout_ns(0)
        _, word = call(dd, R, s, ws=ws, state_out=torch.empty_like(to))
        assert word == ms.ETIMEOUT
    finally:
        ms.set_wait_timeout_ns(2_000_000_000)
    out = torch.zeros_like(a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ms.block_delta_rule(dd, R, s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], out, ws, state_out=to, qk_eps=1e-6)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, out) and torch.equal(first[:R], to[:R])


@pytest.mark.parametrize("dtype,step", [(ms.F32, 3000), (ms.F32, 1), (ms.BF16, 3000), (ms.BF16, 1), (ms.BF16, 32)])
def test_slow_decays_do_not_drift(dtype, step):
    """Thousands of decays close to 1, in one call, in blocks and token by token: the state is multiplied by each, and the
    errors of their roundings must not all point the same way.  With beta = 0 it ends as its start times e^(sum of g).  A
    factor and a product are each off by 2^-25 of a value at most (values in [1/2, 1)) or 2^-24 in all, uniformly, so with a
    standard deviation of 2^-24 / sqrt(3) a token; six of them after n tokens are allowed."""
    n = 3000 if step != 32 else 3008
    dd = ms.DeltaDims(Hk=1, Hv=2, Dk=64, Dv=64, n_slots=1, dtype=dtype)
    s = make(dd, 1, n, 7)
    g = torch.Generator(device="cuda").manual_seed(8)
    s["g"] = -2e-4 * torch.exp(0.5 * torch.randn((n, 2), generator=g, device="cuda"))
    s["beta"].zero_()
    start, ws = s["state"].clone(), ms.delta_workspace(dd, 1, step)
    out = torch.empty((step, 2, 64), device="cuda", dtype=s["q"].dtype)
    for t in range(0, n, step):
        ms.block_delta_rule(dd, 1, s["q"][t:t + step], s["k"][t:t + step], s["v"][t:t + step], s["g"][t:t + step],
                            s["beta"][t:t + step], s["state"], out, ws, state_out=s["state"], qk_eps=1e-6)
    torch.cuda.synchronize()
    assert ms.read_device_error(ws) == ms.OK
    want = start.double() * torch.exp(s["g"].double().sum(0))[None, :, None, None]
    off = ((s["state"].double() - want).norm(dim=-1) / want.norm(dim=-1)).max()
    assert off <= 6 * n ** 0.5 * 2.0 ** -24 / 3 ** 0.5, float(off)
