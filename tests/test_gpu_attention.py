"""block_attention against the float64 oracle.

Bounds, elementwise, with wabs = sum_j p_j |v_j| and u = 2^-24 (the oracle returns wabs and
dots = max_j scale * sum_d |q_d k_jd|):

* scores: D products summed in fp32, twice u a step (truncating adders included), and the
  scale: |ds| <= (D + 4) 2 u dots =: e;  the argument's rounding in the exponential 4 u (dots + 20);
* weights: relative error e + 4 u (dots + 20) + 2^-21 (the exponential), twice that after the division;
* sums over n keys: n 2 u at most;
* bf16 and fp8 caches: each weight rounds once to bf16, 2^-8 relative, and so does the output.

so |d out| <= wabs (2 e + 8 u (dots + 20) + 2^-20 + 2 n u + [2^-8]) + |out| [2^-8] or u, and
|d lse| <= e + 4 u (dots + 20) + 2^-20 + 2 n u + 2 u |lse|."""
import numpy as np
import pytest
import torch

import moe_expert_step_gb300 as ms
from oracle import kv_attention as KV

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
ACT = {ms.BF16: torch.bfloat16, ms.FP8: torch.bfloat16, ms.F32: torch.float32}
KIND = [ms.BF16, ms.F32, ms.FP8]
NAN8 = 0x7F


class Setup:
    """Requests of the given lengths in a shuffled pool.  Every place that no query may use holds
    NaN, and every table entry that no query needs points outside the pool."""

    def __init__(self, dtype, lengths, n_q, Hkv, G, D, page, window=0, seed=0, strided=False, spread=1.0):
        g = np.random.default_rng(seed)
        self.dtype, self.lengths, self.n_q, self.window = dtype, lengths, n_q, window
        R, Hq = len(lengths), Hkv * G
        self.R, self.scale = R, D ** -0.5
        max_pages = max(1, max(-(-L // page) for L in lengths)) + 1
        used = sum(-(-L // page) for L in lengths)
        n_pages = used + 2
        order, at = g.permutation(n_pages).astype(np.int32), 0
        table = np.full((R, max_pages), n_pages + 7, np.int32)
        table[:, 1::2] = -1
        pools = [torch.full((n_pages, Hkv, page, D), float("nan")) for _ in "kv"]
        exps = [torch.full((n_pages, Hkv, page), 255, dtype=torch.uint8) for _ in "kv"]
        self.k, self.v = [], []
        for r, L in enumerate(lengths):
            lo = max(0, L - n_q - window + 1) if window else 0
            for store, pool, ex in ((self.k, pools[0], exps[0]), (self.v, pools[1], exps[1])):
                x = (spread * g.standard_normal((L, Hkv, D)) * np.exp(0.4 * g.standard_normal((L, Hkv, 1)))).astype(np.float32)
                if dtype != ms.F32:
                    x = torch.from_numpy(x).bfloat16().float().numpy()
                store.append(x)
            for p0 in range(0, L, page):
                if p0 + page <= lo:
                    continue
                if table[r, p0 // page] == n_pages + 7 or table[r, p0 // page] == -1:
                    table[r, p0 // page] = order[at]
                    at += 1
                n = min(page, L - p0)
                a = max(lo - p0, 0)
                for store, pool, ex in ((self.k, pools[0], exps[0]), (self.v, pools[1], exps[1])):
                    x = store[r][p0 + a:p0 + n]
                    if dtype == ms.FP8:
                        q = np.empty_like(x)
                        for i in range(x.shape[0]):
                            for h in range(Hkv):
                                qq, e = KV.quantise(x[i, h])
                                q[i, h] = qq
                                store[r][p0 + a + i, h] = qq * 2.0 ** e
                                ex[table[r, p0 // page], h, a + i] = e + 127
                        x = q
                    pool[table[r, p0 // page], :, a:n] = torch.from_numpy(x).transpose(0, 1)
        cast = {ms.BF16: torch.bfloat16, ms.F32: torch.float32, ms.FP8: torch.float8_e4m3fn}[dtype]
        pools = [p.to(cast).cuda() for p in pools]
        exps = [e.cuda() if dtype == ms.FP8 else None for e in exps]
        self.table = torch.from_numpy(table).cuda()
        self.kd = ms.KvDims(Hq=Hq, Hkv=Hkv, D=D, page=page, n_pages=n_pages, max_pages=max_pages, dtype=dtype)
        self.pools = pools
        self.cache = ms.kv_cache(*pools, self.table, *exps)
        self.len = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        T = R * n_q
        q = torch.from_numpy((1.5 * g.standard_normal((T, Hq + 2, D))).astype(np.float32)).to(ACT[dtype]).cuda()
        self.q = q[:, 1:1 + Hq] if strided else q[:, :Hq].contiguous()
        self.ws = ms.kv_workspace(self.kd, R, n_q)

    def run(self, causal=False, lse=True, stream=None):
        out = torch.full(self.q.shape, 7.0, dtype=self.q.dtype, device="cuda")
        ls = torch.full(self.q.shape[:2], 7.0, device="cuda") if lse else None
        ms.block_attention(self.kd, self.R, self.q, self.len, self.cache, out, self.ws, self.scale, causal=causal,
                           window=self.window, lse=ls, stream=stream)
        return out, ls

    def check(self, out, ls, causal=False):
        torch.cuda.synchronize()
        assert ms.read_device_error(self.ws) == ms.OK
        o, l, wabs, dots = KV.block_attention(self.q.float().cpu().numpy(), self.k, self.v, self.lengths, self.n_q,
                                              np.float32(self.scale), causal, self.window)
        n = max(max(self.lengths), 1)
        e = (self.kd.D + 4) * 2 * U * dots
        half = U if self.dtype == ms.F32 else 2.0 ** -8
        arg = 4 * U * (dots + 20)
        rel = 2 * e + 2 * arg + 2.0 ** -20 + 2 * n * U + (0 if self.dtype == ms.F32 else half)
        bound = wabs * rel[..., None] * 1.01 + np.abs(o) * half * 1.01 + 1e-30
        got = out.float().cpu().numpy()
        assert np.isfinite(got).all()
        worst = (np.abs(got - o) / bound).max()
        assert worst <= 1, worst
        if ls is not None:
            gl = ls.cpu().numpy()
            empty = np.isneginf(l)
            assert (np.isneginf(gl) == empty).all()
            lb = e + arg + 2.0 ** -20 + 2 * n * U + 2 * U * np.abs(np.where(empty, 0, l))
            assert (np.abs(gl - l)[~empty] <= lb[~empty]).all()
        return worst


SHAPES = [  # lengths, n_q, Hkv, G, D, page
    ([1], 1, 1, 1, 64, 16),
    ([5, 0, 130, 64], 1, 2, 8, 128, 16),
    ([127, 128, 129, 255, 256, 257], 1, 1, 4, 128, 32),
    ([300], 32, 2, 8, 128, 64),
    ([33, 0, 700], 32, 1, 2, 64, 16),
    ([100, 3], 5, 2, 3, 64, 128),
    ([2000], 1, 1, 16, 128, 64),
    ([513, 40], 16, 1, 6, 128, 128),
    ([260], 64, 1, 5, 64, 32),
    ([1, 1, 1], 3, 2, 1, 128, 16),
    ([390], 33, 1, 4, 128, 16),
    ([129], 129, 1, 2, 64, 64),
]


@pytest.mark.parametrize("dtype", KIND)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("causal", [False, True])
def test_against_the_oracle(dtype, shape, causal):
    s = Setup(dtype, *shape)
    s.check(*s.run(causal), causal)


@pytest.mark.parametrize("dtype", KIND)
@pytest.mark.parametrize("window", [1, 7, 16, 100, 128, 1000])
@pytest.mark.parametrize("causal", [False, True])
def test_window(dtype, window, causal):
    s = Setup(dtype, [400, 17, 0, 128], 9, 2, 2, 64, 16, window=window, strided=True)
    s.check(*s.run(causal), causal)


@pytest.mark.parametrize("dtype", KIND)
def test_long_ragged_batch(dtype):
    """Many segments that CTAs share, beside whole ones and idle slots."""
    s = Setup(dtype, [3500, 1, 0, 0, 1777, 64, 900, 2], 1, 2, 4, 64, 64, seed=5)
    s.check(*s.run())
    s = Setup(dtype, [2500, 12, 0, 1300], 8, 1, 8, 128, 32, seed=6)
    s.check(*s.run(True), True)


@pytest.mark.parametrize("dtype", KIND)
def test_large_scores(dtype):
    """Scores far apart: the running maximum moves by hundreds, one key takes nearly all the weight."""
    s = Setup(dtype, [600, 40], 4, 1, 2, 64, 16, spread=30.0, seed=7)
    s.check(*s.run())


@pytest.mark.parametrize("dtype", KIND)
def test_growing_scores(dtype):
    """Every tile brings a new maximum."""
    s = Setup(dtype, [1500], 2, 1, 4, 128, 64, seed=8)
    torch.cuda.synchronize()
    q = s.q.float().mean(0, keepdim=True).expand_as(s.q)
    s.q = q.to(s.q.dtype).contiguous()
    order = np.argsort(s.k[0][:, 0] @ s.q.float().cpu().numpy()[0, 0])
    s.k[0] = s.k[0][order]
    tab = s.table.cpu().numpy()[0]
    ids = torch.from_numpy(tab[np.arange(1500) // 64].astype(np.int64))
    at = torch.arange(1500) % 64
    flat = (ids * 64 + at).cuda()
    o = torch.from_numpy(order).cuda()
    for t in (s.pools[0].view(torch.uint8 if dtype == ms.FP8 else s.pools[0].dtype), s.cache._tensors[3]):
        if t is not None:
            rows = t.reshape(-1, t.shape[-1]) if t.dim() == 4 else t.reshape(-1)
            rows[flat] = rows[flat][o]
    s.check(*s.run())


@pytest.mark.parametrize("dtype", KIND)
def test_repeats_and_streams(dtype):
    """The same bits on every call, on another stream, without lse, and replayed from a graph."""
    s = Setup(dtype, [1900, 50, 333], 4, 2, 4, 128, 32, seed=9)
    out, ls = s.run(True)
    for _ in range(3):
        o2, l2 = s.run(True)
        assert torch.equal(out, o2) and torch.equal(ls, l2)
    assert torch.equal(out, s.run(True, lse=False)[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o3, _ = s.run(True)
    side.synchronize()
    assert torch.equal(out, o3)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o4, _ = s.run(True)
    s.len.copy_(torch.tensor([7, 50, 0], dtype=torch.int32))     # lengths are read when it runs
    g.replay()
    s.lengths = [7, 50, 0]
    s.k, s.v = ([x[:n] for x, n in zip(t, s.lengths)] for t in (s.k, s.v))
    s.check(o4, None, True)
    s.len.copy_(torch.tensor([1900, 50, 333], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o4, out)


@pytest.mark.parametrize("n_q", [1, 17])
@pytest.mark.parametrize("dtype", [ms.BF16, ms.FP8])
def test_many_one_tile_segments_of_a_cta(dtype, n_q):
    """Several requests of one key tile each in a row on every CTA: each role goes from segment to
    segment with the others up to a ring of buffers ahead."""
    lengths = [n_q + (7 * r) % 23 for r in range(400 if n_q == 1 else 200)]
    s = Setup(dtype, lengths, n_q, Hkv=2, G=8, D=128, page=16, seed=3)
    out, ls = s.run()
    s.check(out, ls)
    for _ in range(20):
        o2, l2 = s.run()
        assert torch.equal(o2, out) and torch.equal(l2, ls)



@pytest.mark.parametrize("dtype", KIND)
def test_many_requests(dtype):
    """More requests than threads of a block: the division of the work scans them in runs."""
    lengths = [(7 * r) % 40 for r in range(700)]
    s = Setup(dtype, lengths, 1, 1, 2, 64, 16, seed=10)
    s.check(*s.run())


@pytest.mark.parametrize("dtype", KIND)
def test_bad_lengths_and_pages_are_reported(dtype):
    """Out-of-range lengths are clamped and pages outside the pool never followed; other requests
    keep their results."""
    s = Setup(dtype, [100, 60, 90], 2, 1, 2, 64, 16, seed=11)
    good, _ = s.run()
    torch.cuda.synchronize()
    s.table[1, 0] = 1 << 30
    s.table[1, 2] = -1
    out, _ = s.run()
    torch.cuda.synchronize()
    assert ms.read_device_error(s.ws) == ms.EDEVINPUT
    assert torch.equal(out[:2], good[:2]) and torch.equal(out[4:], good[4:])
    s.len.copy_(torch.tensor([100, -3, 1 << 30], dtype=torch.int32))
    out, ls = s.run()
    torch.cuda.synchronize()
    assert ms.read_device_error(s.ws) == ms.EDEVINPUT
    assert torch.equal(out[:2], good[:2]) and not out[2:4].any() and torch.isneginf(ls[2:4]).all()


def test_offsets_past_32_bits():
    """Pages beyond 2^32 elements of the pool give what the same pages give at its start."""
    n_pages = (1 << 32) // (8 * 128 * 128) + 40
    kd = ms.KvDims(Hq=16, Hkv=8, D=128, page=128, n_pages=n_pages, max_pages=3, dtype=ms.BF16)
    k = torch.empty((n_pages, 8, 128, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    for t in (k, v):
        t[:3].normal_()
        t[n_pages - 3:] = t[:3]
    q = torch.randn((4, 16, 128), device="cuda").bfloat16()
    n = torch.tensor([300], dtype=torch.int32, device="cuda")
    ws, outs = ms.kv_workspace(kd, 1, 4), []
    for first in (0, n_pages - 3):
        c = ms.kv_cache(k, v, torch.arange(first, first + 3, dtype=torch.int32, device="cuda")[None].contiguous())
        outs.append(torch.empty_like(q))
        ms.block_attention(kd, 1, q, n, c, outs[-1], ws, 0.09)
    torch.cuda.synchronize()
    assert ms.read_device_error(ws) == ms.OK and torch.equal(*outs) and torch.isfinite(outs[0].float()).all()


@pytest.mark.parametrize("dtype", [ms.BF16, ms.FP8])
@pytest.mark.parametrize("shape", [([700, 40, 0], 1, 2, 4, 128, 32), ([900, 300], 32, 1, 8, 128, 64),
                                   ([500], 16, 1, 4, 64, 16), ([400], 32, 1, 4, 64, 128)])
def test_wait_timeout_is_reported_and_recovered(dtype, shape):
    """A limit of zero makes the kernel's bounded waits give up; it drains what it issued, reports,
    and the next call is right."""
    s = Setup(dtype, *shape, seed=12)
    good, _ = s.run()
    torch.cuda.synchronize()
    try:
        ms.set_wait_timeout_ns(0)
        s.run()
        assert ms.read_device_error(s.ws) == ms.ETIMEOUT
    finally:
        ms.set_wait_timeout_ns(2_000_000_000)
    out, ls = s.run()
    assert torch.equal(out, good)
    s.check(out, ls)


@pytest.mark.parametrize("dtype", KIND)
def test_nan_where_it_is_seen(dtype):
    """NaN in a visible key or value reaches its own head's rows and no others; an infinite query
    its own row."""
    s = Setup(dtype, [300, 77], 2, 2, 2, 64, 16, seed=13)
    good, _ = s.run()
    tab = s.table.cpu().numpy()
    for pool in s.pools:                                   # one of the two at a time
        raw = pool.view(torch.uint8) if dtype == ms.FP8 else pool
        at = (int(tab[0, 200 // 16]), 1, 200 % 16, 5)      # request 0, key-value head 1
        old = raw[at].clone()
        raw[at] = 0x7F if dtype == ms.FP8 else float("nan")
        out, _ = s.run()
        raw[at] = old
        bad = torch.isnan(out.float()).any(-1).cpu().numpy()
        assert bad[:2, 2:].all() and not bad[:2, :2].any() and not bad[2:].any()
        assert torch.equal(out[2:], good[2:]) and torch.equal(out[:2, :2], good[:2, :2])
    s.q[1, 3, 7] = float("inf")
    out, _ = s.run()
    bad = torch.isnan(out.float()).any(-1).cpu().numpy()
    assert bad[1, 3] and bad.sum() == 1


@pytest.mark.parametrize("exps", [(-90, -80), (100, 110), (-3, 20)])
def test_fp8_scales_far_from_one(exps):
    """Exponents below and above what one bf16 factor holds: keys and queries scaled so that the
    scores stay moderate, values anywhere."""
    s = Setup(ms.FP8, [400, 33], 3, 1, 2, 128, 32, seed=14)
    g = np.random.default_rng(15)
    ek, ev = s.cache._tensors[3], s.cache._tensors[4]
    tab = s.table.cpu().numpy()
    dv = g.integers(exps[0], exps[1] + 1, 2)
    for r, L in enumerate(s.lengths):
        for j in range(L):
            i = (int(tab[r, j // 32]), 0, j % 32)
            ev[i] = int(ev[i]) + int(dv[r])
            ek[i] = int(ek[i]) + 20
        s.v[r] = s.v[r].astype(np.float64) * 2.0 ** int(dv[r])
        s.k[r] = s.k[r].astype(np.float64) * 2.0 ** 20
    s.q = (s.q.float() * 2.0 ** -20).bfloat16()
    s.check(*s.run())
