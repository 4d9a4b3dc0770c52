"""kv_cache_plan against the plain oracle: every output equal, on rings that wrap, requests that end, are cut back
or refused, and bad values."""
import numpy as np
import pytest
import torch

import moe_expert_step_gb300 as ms
from oracle import token_mixer as om

pytestmark = pytest.mark.gpu

dev = lambda a: torch.as_tensor(np.ascontiguousarray(a)).to(torch.int32).cuda()  # noqa: E731


def make(R, n, page, seed, spare=4, drop=0.25, length=None):
    """Requests holding pages of their own, the others free in a ring that begins anywhere."""
    rng = np.random.default_rng(seed)
    length = 5 * page if length is None else length
    kv_len = rng.integers(0, length + 1, R)
    n_new = rng.integers(0, n + 1, R)
    ends, cut = rng.random(R) < drop / 2, rng.random(R) < drop / 2
    n_new = np.where(ends, -kv_len, np.where(cut, -np.minimum(kv_len, rng.integers(0, n + 1, R)), n_new))
    max_pages = -(-(length + n) // page)
    held = -(-kv_len // page)
    grow = np.maximum(0, -(-(kv_len + n_new) // page) - held)
    free = max(0, int(grow.sum()) + spare)
    n_pages = max(1, int(held.sum()) + free)
    order = rng.permutation(n_pages)
    table = np.full((R, max_pages), -1)
    at = 0
    for r in range(R):
        table[r, :held[r]] = order[at:at + held[r]]
        at += held[r]
    first = int(rng.integers(0, n_pages))
    ring = np.full(n_pages, -7)
    ring[(first + np.arange(n_pages - at)) % n_pages] = order[at:]
    kd = ms.KvDims(Hq=4, Hkv=2, D=64, page=page, n_pages=n_pages, max_pages=max_pages)
    return kd, kv_len, n_new, ring, np.array([first, n_pages - at]), table


def call(kd, kv_len, n_new, ring, head, table, n, ws=None, in_place=False, slots=True, stream=None):
    R = len(kv_len)
    t = dict(kv_len=dev(kv_len), n_new=dev(n_new), ring=dev(ring), head=dev(head), table=dev(table))
    out = torch.full((2,), -9, dtype=torch.int32, device="cuda")
    head_out = t["head"] if in_place else out
    new_len, pos = dev(np.full(R, -9)), dev(np.full((R, n), -9))
    sl = dev(np.full((R, n), -9)) if slots else None
    ws = ms.kv_workspace(kd, R, 1) if ws is None else ws
    ms.kv_cache_plan(kd, R, t["kv_len"], t["n_new"], t["ring"], t["head"], head_out, t["table"], new_len, pos, ws,
                     slots=sl, stream=stream)
    torch.cuda.synchronize()
    got = [t["ring"], head_out, t["table"], new_len, pos] + ([sl] if slots else [])
    return [x.cpu().numpy() for x in got], ms.read_device_error(ws)


def check(got, want):
    for name, a, b in zip(("ring", "head", "table", "new_len", "pos", "slots"), got, want):
        np.testing.assert_array_equal(a, b, err_msg=name)


@pytest.mark.parametrize("R,n,page", [(1, 1, 16), (1, 32, 64), (2, 7, 16), (5, 33, 32), (3, 4096, 128), (2, 9001, 16),
                                      (300, 5, 16), (257, 1, 64), (700, 40, 32), (4100, 1, 16), (17, 4095, 64)])
@pytest.mark.parametrize("spare", [3, 0, -1, -40])
def test_against_oracle(R, n, page, spare):
    kd, *state = make(R, n, page, R * 31 + n, spare)
    want = om.kv_cache_plan(state[0], state[1], n, *state[2:], page)
    got, word = call(kd, *state, n, in_place=spare == 0)
    check(got, want)
    assert word == ms.OK


def test_calls_follow_each_other():
    """Blocks of 32 positions after one another, requests ending and starting again, in place, without slots; no page
    is ever held twice."""
    R, n, page = 40, 32, 16
    kd, kv_len, _, ring, head, table = make(R, n, page, 5, spare=200)
    rng = np.random.default_rng(6)
    ws = ms.kv_workspace(kd, R, 1)
    for _ in range(12):
        n_new = np.where(rng.random(R) < 0.2, -kv_len, rng.integers(0, n + 1, R))
        want = om.kv_cache_plan(kv_len, n_new, n, ring, head, table, page)
        got, word = call(kd, kv_len, n_new, ring, head, table, n, ws=ws, in_place=True, slots=False)
        check(got, want)
        assert word == ms.OK
        ring, head, table, kv_len = (np.array(x) for x in want[:4])
        free = ring[(head[0] + np.arange(head[1])) % len(ring)]
        held = np.concatenate([table[r, :-(-kv_len[r] // page)] for r in range(R)])
        assert len(np.unique(np.concatenate([free, held]))) == len(free) + len(held)


def test_positions_as_the_cache_takes_them():
    """Tokens written at the planned positions are read back from the planned slots."""
    R, n, page = 6, 37, 16
    kd, *state = make(R, n, page, 11, drop=0.0)
    got, word = call(kd, *state, n)
    assert word == ms.OK
    _, _, table, new_len, pos, slots = got
    k, v = (torch.randn((R * n, 2, 64), device="cuda").bfloat16() for _ in "kv")
    pool = [torch.zeros((kd.n_pages, 2, page, 64), device="cuda").bfloat16() for _ in "kv"]
    cache, ws = ms.kv_cache(*pool, dev(table)), ms.kv_workspace(kd, R, 1)
    ms.kv_cache_write(kd, R, k, v, dev(pos), cache, ws)
    assert ms.read_device_error(ws) == ms.OK
    at = torch.as_tensor(slots.reshape(-1)).cuda().long()
    rows = pool[0].transpose(1, 2).reshape(-1, 2, 64)
    assert torch.equal(rows[at[at >= 0]], k[at >= 0])
    np.testing.assert_array_equal(new_len, np.asarray(state[0]) + np.asarray(state[1]))


@pytest.mark.parametrize("what", ["len_negative", "len_long", "new_long", "new_negative", "past_table", "page", "gone_page",
                                  "first", "count", "too_many"])
def test_bad_values_are_recorded(what):
    """A request with a value out of range is refused, the others are served; nothing is followed."""
    R, n, page = 5, 20, 16
    kd, kv_len, n_new, ring, head, table = make(R, n, page, 3, drop=0.0, spare=5)
    kv_len[2], n_new[2] = 30, 10  # two pages held, one more
    kd, kv_len, n_new, ring, head, table = rebuild(kv_len, n_new, n, page)
    bad = ms.EDEVINPUT
    skip = True
    if what == "len_negative":
        kv_len[2] = -1
    elif what == "len_long":
        kv_len[2] = kd.max_pages * page + 1
    elif what == "new_long":
        n_new[2] = n + 1
    elif what == "new_negative":
        n_new[2] = -31
    elif what == "past_table":
        kv_len[2] = kd.max_pages * page - 3  # a refusal, not an error
        bad = ms.OK
    else:
        skip = False
    if skip:
        want = om.kv_cache_plan(kv_len, n_new, n, ring, head, table, page)
    if what == "page":
        ring[head[0] % len(ring)] = kd.n_pages
    elif what == "gone_page":
        n_new[2], table[2, 1] = -20, -5
    elif what == "first":
        head[0] = kd.n_pages
    elif what == "count":
        head[1] = kd.n_pages + 1
    elif what == "too_many":  # the ring says that it is full, and pages come back
        head[1], n_new[:] = kd.n_pages, -kv_len
    got, word = call(kd, kv_len, n_new, ring, head, table, n)
    assert word == bad
    if skip:
        check(got, want)
    if what in ("first", "count"):
        np.testing.assert_array_equal(got[1], head)
        np.testing.assert_array_equal(got[0], ring)
        assert (got[4] < 0).any()
    if what == "page":
        assert (got[2] == -1).any() and got[5].max() < kd.n_pages * page
    if what == "too_many":
        assert got[1][1] == kd.n_pages


def rebuild(kv_len, n_new, n, page):
    held = -(-kv_len // page)
    max_pages = -(-(kv_len.max() + n) // page) + 1
    n_pages = int(held.sum()) + 12
    table = np.full((len(kv_len), max_pages), -1)
    at = 0
    for r, h in enumerate(held):
        table[r, :h] = np.arange(at, at + h)
        at += h
    ring = np.full(n_pages, -7)
    ring[(n_pages - 4 + np.arange(12)) % n_pages] = np.arange(at, at + 12)
    kd = ms.KvDims(Hq=4, Hkv=2, D=64, page=page, n_pages=n_pages, max_pages=int(max_pages))
    return kd, np.array(kv_len), np.array(n_new), ring, np.array([n_pages - 4, 12]), table


def test_captured_and_on_another_stream():
    R, n, page = 300, 50, 16
    kd, *state = make(R, n, page, 21)
    want = om.kv_cache_plan(state[0], state[1], n, *state[2:], page)
    s = torch.cuda.Stream()
    ws = ms.kv_workspace(kd, R, 1)
    torch.cuda.synchronize()
    got, word = call(kd, *state, n, ws=ws, stream=s)
    check(got, want)
    t = [dev(x) for x in state]
    keep = [x.clone() for x in t]
    head_out, new_len, pos, slots = (torch.zeros(k, dtype=torch.int32, device="cuda") for k in ((2,), (R,), (R, n), (R, n)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ms.kv_cache_plan(kd, R, t[0], t[1], t[2], t[3], head_out, t[4], new_len, pos, ws, slots=slots)
    for _ in range(2):
        for a, b in zip(t, keep):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        check([x.cpu().numpy() for x in (t[2], head_out, t[4], new_len, pos, slots)], want)
    assert ms.read_device_error(ws) == ms.OK
