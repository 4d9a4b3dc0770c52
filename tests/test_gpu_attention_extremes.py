"""block_attention where scores pass 2^30, so that fp32 holds no fraction of them: the softmax is one key's, or
some equal ones', or that of the keys whose scores are moderate beside huge negative ones.

Bounds.  A weight of 1 is rounded to bf16 beside a sum that is not (2^-8), the output too (2^-8), fp32 adds
2^-20.  Scores: D products summed in fp32 and four roundings, (D + 8) 2 u of sum |q_d k_d|, with FP8 caches
also 2^-17 of the row's largest query element times sum |k_d| (the split of the queries).  Among the moderate
keys as in test_gpu_attention.py, with those scores' bound."""
import numpy as np
import pytest
import torch

import moe_expert_step_gb300 as ms
from oracle import kv_attention as KV

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
KIND = [ms.BF16, ms.F32, ms.FP8]
L, PAGE, G = 300, 32, 2
STORE = {ms.BF16: torch.bfloat16, ms.F32: torch.float32, ms.FP8: torch.float8_e4m3fn}


def attend(dtype, k, v, q, R):
    """R requests of the same queries [n_q, G, D] over the same pages: the stored keys and values, the queries
    as passed, and one request's results (all have to be equal)."""
    D, n_q = k.shape[1], q.shape[0]
    act = torch.float32 if dtype == ms.F32 else torch.bfloat16
    pages = -(-L // PAGE)
    kd = ms.KvDims(Hq=G, Hkv=1, D=D, page=PAGE, n_pages=pages, max_pages=pages, dtype=dtype)
    pools = [torch.zeros((pages, 1, PAGE, D), device="cuda").to(STORE[dtype]) for _ in "kv"]
    exps = [torch.zeros((pages, 1, PAGE), dtype=torch.uint8, device="cuda") if dtype == ms.FP8 else None for _ in "kv"]
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda().repeat(R, 1)
    cache, ws = ms.kv_cache(*pools, table, *exps), ms.kv_workspace(kd, R, n_q)
    pos = torch.arange(L, dtype=torch.int32, device="cuda")[None]
    new = [torch.from_numpy(x).to(act).cuda()[:, None] for x in (k, v)]
    ms.kv_cache_write(kd, 1, *new, pos, cache, ws)
    back = [torch.empty_like(x) for x in new]
    ms.kv_cache_read(kd, 1, pos, cache, *back, ws)
    qs = torch.from_numpy(q).to(act).cuda().repeat(R, 1, 1)
    out, lse = torch.empty_like(qs), torch.empty((R * n_q, G), device="cuda")
    n = torch.full((R,), L, dtype=torch.int32, device="cuda")
    ms.block_attention(kd, R, qs, n, cache, out, ws, D ** -0.5, lse=lse)
    torch.cuda.synchronize()
    assert ms.read_device_error(ws) == ms.OK
    out, lse = out.view(R, n_q, G, D), lse.view(R, n_q, G)
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    f = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
    return (*(f(b)[:, 0] for b in back), f(qs[:n_q]), f(out), f(lse))


def score_error(dtype, q, k):
    """[n_q, G] bound of the scores' errors over the keys."""
    D = k.shape[1]
    e = (D + 8) * 2 * U * (np.abs(q) @ np.abs(k).T).max(-1)
    if dtype == ms.FP8:
        e += 2.0 ** -17 * np.abs(q).max(-1) * np.abs(k).sum(-1).max()
    return np.float32(D ** -0.5) * e


def direction(D, n_q, seed):
    """A direction and queries along it, of three lengths about 2^20."""
    g = np.random.default_rng(seed)
    u = torch.from_numpy(g.standard_normal(D)).bfloat16().double().numpy()
    a = 2.0 ** (20 + g.integers(-1, 2, (n_q, G)))
    return g, u, a[..., None] * u


@pytest.mark.parametrize("R", [1, 120])
@pytest.mark.parametrize("n_q,D", [(3, 64), (3, 128), (20, 128), (50, 64), (80, 128)])
@pytest.mark.parametrize("dtype", KIND)
@pytest.mark.parametrize("sign", [1, -1])
def test_one_key_of_huge_scores(dtype, n_q, D, R, sign):
    """The largest score is 2^43 and a quarter above the next, or all are negative and it is as much nearer to 0;
    then three equal keys share it."""
    g, u, q = direction(D, n_q, 40)
    c = g.uniform(-1, 0.75, L) if sign > 0 else g.uniform(-1, -0.5, L)
    v = g.standard_normal((L, D))
    for best in ([101], [30, 101, 290]):
        c[best] = 1.0 if sign > 0 else -0.375
        ks, vs, qs, out, lse = attend(dtype, 2.0 ** 20 * c[:, None] * u, v, q, R)
        want = vs[best].mean(0)
        s = np.float32(D ** -0.5) * (qs @ ks[best[0]])
        bound = (2.0 ** -20 if dtype == ms.F32 else 2.0 ** -7) * np.abs(vs[best]).mean(0) * 1.01
        assert (np.abs(out - want) <= bound).all()
        assert (np.abs(lse - s) <= score_error(dtype, qs, ks[best]) + 4 * U * np.abs(s) + 1).all()


@pytest.mark.parametrize("R", [1, 120])
@pytest.mark.parametrize("n_q,D", [(3, 64), (3, 128), (20, 128), (50, 64), (80, 128)])
@pytest.mark.parametrize("dtype", KIND)
@pytest.mark.parametrize("where", ["first", "last", "between"])
def test_moderate_scores_beside_huge_negative_ones(dtype, where, n_q, D, R):
    g, u, q = direction(D, n_q, 41)
    j = np.arange(L)
    huge = j < 200 if where == "first" else j >= 40 if where == "last" else (j // 8) % 2 == 0
    k = np.where(huge[:, None], -2.0 ** 20 * g.uniform(0.5, 1, (L, 1)) * u, 2.0 ** -20 * g.standard_normal((L, D)))
    ks, vs, qs, out, lse = attend(dtype, k, g.standard_normal((L, D)), q, R)
    km, vm = ks[~huge], vs[~huge]
    o, l, wabs, dots = KV.block_attention(qs, [km[:, None]], [vm[:, None]], [len(km)], n_q, np.float32(D ** -0.5), False, 0)
    e = score_error(dtype, qs, km)
    arg = 4 * U * (dots + 20)
    half = U if dtype == ms.F32 else 2.0 ** -8
    rel = 2 * e + 2 * arg + 2.0 ** -20 + 2 * L * U + (0 if dtype == ms.F32 else half)
    assert (np.abs(out - o) <= wabs * rel[..., None] * 1.01 + np.abs(o) * half * 1.01).all()
    assert (np.abs(lse - l) <= e + arg + 2.0 ** -20 + 2 * L * U + 2 * U * np.abs(l)).all()
