"""kv_cache_write / kv_cache_read against the oracle: codes, exponents and copies are exact."""
import numpy as np
import pytest
import torch

import moe_expert_step_gb300 as ms
from oracle import kv_attention as KV

pytestmark = pytest.mark.gpu
ACT = {ms.BF16: torch.bfloat16, ms.FP8: torch.bfloat16, ms.F32: torch.float32}
STORE = {ms.BF16: torch.bfloat16, ms.FP8: torch.float8_e4m3fn, ms.F32: torch.float32}
KIND = [ms.BF16, ms.F32, ms.FP8]


def make(dtype, R, Hkv, D, page, max_pages, n_pages, seed=0):
    """An empty cache (zeros), its pages dealt out at random."""
    kd = ms.KvDims(Hq=Hkv, Hkv=Hkv, D=D, page=page, n_pages=n_pages, max_pages=max_pages, dtype=dtype)
    g = np.random.default_rng(seed)
    table = torch.from_numpy(g.permutation(n_pages)[:R * max_pages].reshape(R, max_pages).astype(np.int32)).cuda()
    pool = lambda: torch.zeros((n_pages, Hkv, page, D), dtype=torch.float32, device="cuda").to(STORE[dtype])  # noqa: E731
    e = [torch.zeros((n_pages, Hkv, page), dtype=torch.uint8, device="cuda") if dtype == ms.FP8 else None for _ in "kv"]
    k, v = pool(), pool()
    return kd, ms.kv_cache(k, v, table, *e), (k, v, *e, table), ms.kv_workspace(kd, R, 1)


def vectors(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda") * torch.exp(3 * torch.randn(shape[:-1] + (1,), generator=g, device="cuda"))
    return x.to(ACT[dtype])


def expect(x, dtype):
    """What is stored of one vector: (values, exponent byte or None)."""
    if dtype != ms.FP8:
        return x, None
    q, e = KV.quantise(x)
    return q, e + 127


@pytest.mark.parametrize("dtype", KIND)
@pytest.mark.parametrize("R,n,Hkv,D,page", [(1, 1, 1, 64, 16), (1, 32, 2, 128, 64), (3, 37, 4, 64, 32),
                                            (2, 5, 8, 128, 128), (2, 33, 3, 128, 16)])
def test_write_then_read(dtype, R, n, Hkv, D, page):
    max_pages = 3 + n // page
    kd, c, (k, v, ke, ve, table), ws = make(dtype, R, Hkv, D, page, max_pages, R * max_pages + 2)
    kv = vectors((R * n, 2 * Hkv + 1, D), dtype, 7)              # rows wider than what is stored
    kn, vn = kv[:, :Hkv], kv[:, Hkv:2 * Hkv]
    first = page - 1                                             # straddles pages, ends inside one
    pos = torch.arange(first, first + n, dtype=torch.int32, device="cuda").repeat(R, 1)
    if n > 2:
        pos[R - 1, n // 2] = -1
        pos[0, :2] = pos[0, :2].flip(0)                          # not in order
    before = [t.clone() if t is not None else None for t in (k, v, ke, ve)]
    ms.kv_cache_write(kd, R, kn, vn, pos, c, ws)
    torch.cuda.synchronize()
    assert ms.read_device_error(ws) == ms.OK
    tab, ps = table.cpu().numpy(), pos.cpu().numpy()
    want = [b.float().cpu().numpy().astype(np.float64) for b in before[:2]]
    wexp = [b.cpu().numpy() if b is not None else None for b in before[2:]]
    dense = []
    for which, new in enumerate((kn, vn)):
        x = new.float().cpu().numpy()
        back = np.zeros((R * n, Hkv, D))
        for t in range(R * n):
            p = ps[t // n, t % n]
            if p < 0:
                continue
            for h in range(Hkv):
                q, e = expect(x[t, h], dtype)
                want[which][tab[t // n, p // page], h, p % page] = q
                back[t, h] = q if e is None else q * 2.0 ** (e - 127)
                if e is not None:
                    wexp[which][tab[t // n, p // page], h, p % page] = e
        dense.append(back)
    for got, w in zip((k, v), want):
        np.testing.assert_array_equal(got.float().cpu().numpy(), w)
    for got, w in zip((ke, ve), wexp):
        if w is not None:
            np.testing.assert_array_equal(got.cpu().numpy(), w)
    ko, vo = (torch.full((R * n, Hkv, D), 9.0, dtype=ACT[dtype], device="cuda") for _ in "kv")
    ms.kv_cache_read(kd, R, pos, c, ko, vo, ws)
    torch.cuda.synchronize()
    assert ms.read_device_error(ws) == ms.OK
    for got, w in zip((ko, vo), dense):                          # code * 2^e is exact in bf16
        np.testing.assert_array_equal(got.float().cpu().numpy(), w)


def test_fp8_special_vectors():
    """Ties, zeros, tiny and huge values, NaN and infinities, against the oracle's rounding."""
    kd, c, (k, v, ke, ve, table), ws = make(ms.FP8, 1, 1, 64, 16, 2, 4)
    rows = torch.randn((20, 1, 64), generator=torch.Generator().manual_seed(3))
    rows[0] = 0.0
    rows[1] *= 1e-36
    rows[2] *= 1e37
    rows[3, 0, 5] = float("nan")
    rows[4, 0, 6], rows[4, 0, 7] = float("inf"), float("-inf")
    rows[5] = torch.arange(64) * 0.0625 + 1.0                     # ties between neighbouring codes
    rows[6] = 448.0
    rows[7] = 449.0
    rows[8] = float("nan")
    rows[9] = 2.0 ** -130
    rows[10] = torch.arange(64) - 32.0
    rows[11, 0, 0] = 3.3e38
    x = rows.bfloat16().cuda()
    pos = torch.arange(20, dtype=torch.int32, device="cuda")[None]
    ms.kv_cache_write(kd, 1, x, -x, pos, c, ws)
    torch.cuda.synchronize()
    tab, xn = table.cpu().numpy()[0], x.float().cpu().numpy()
    for t in range(20):
        for pool, ex, s in ((k, ke, 1.0), (v, ve, -1.0)):
            q, e = KV.quantise(s * xn[t, 0])
            np.testing.assert_array_equal(pool.float().cpu().numpy()[tab[t // 16], 0, t % 16], q, err_msg=str(t))
            assert int(ex[tab[t // 16], 0, t % 16]) == e + 127, t


@pytest.mark.parametrize("dtype", KIND)
def test_bad_places_are_reported_and_not_followed(dtype):
    kd, c, (k, v, ke, ve, table), ws = make(dtype, 2, 2, 64, 16, 3, 8)
    table[1, 0], table[1, 1] = 8, -5                             # outside the pool
    x = vectors((6, 2, 64), dtype, 1)
    pos = torch.tensor([[0, 48, 2 ** 31 - 1], [3, 17, 33]], dtype=torch.int32, device="cuda")
    ms.kv_cache_write(kd, 2, x, x, pos, c, ws)
    torch.cuda.synchronize()
    assert ms.read_device_error(ws) == ms.EDEVINPUT
    touched = k.float().abs().sum((1, 3)).nonzero().cpu().numpy()  # (page, place)
    t = table.cpu().numpy()
    assert {tuple(r) for r in touched} == {(t[0, 0], 0), (t[1, 2], 1)}
    o = [torch.full((6, 2, 64), 9.0, dtype=ACT[dtype], device="cuda") for _ in "kv"]
    ms.kv_cache_read(kd, 2, pos, c, *o, ws)
    torch.cuda.synchronize()
    assert ms.read_device_error(ws) == ms.EDEVINPUT
    assert [bool(r.any()) for r in o[0].float()] == [True, False, False, False, False, True]
    assert ms.read_device_error(ws) == ms.OK


def test_offsets_past_32_bits():
    """A pool of more than 2^32 elements: its last page is written and read back."""
    n_pages = (1 << 32) // (8 * 128 * 128) + 40
    kd = ms.KvDims(Hq=8, Hkv=8, D=128, page=128, n_pages=n_pages, max_pages=2, dtype=ms.BF16)
    k = torch.empty((n_pages, 8, 128, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    table = torch.tensor([[n_pages - 1, 0]], dtype=torch.int32, device="cuda")
    c, ws = ms.kv_cache(k, v, table), ms.kv_workspace(kd, 1, 1)
    x = vectors((3, 16, 128), ms.BF16, 4)
    pos = torch.tensor([[125, 127, 128]], dtype=torch.int32, device="cuda")
    ms.kv_cache_write(kd, 1, x[:, :8], x[:, 8:], pos, c, ws)
    ko, vo = torch.empty((3, 8, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((3, 8, 128), dtype=torch.bfloat16, device="cuda")
    ms.kv_cache_read(kd, 1, pos, c, ko, vo, ws)
    torch.cuda.synchronize()
    assert torch.equal(ko, x[:, :8]) and torch.equal(vo, x[:, 8:])
    assert torch.equal(k[n_pages - 1, :, 127], x[1, :8]) and torch.equal(v[0, :, 0], x[2, 8:])


def test_on_a_stream_of_its_own():
    kd, c, pool, ws = make(ms.BF16, 1, 2, 128, 64, 2, 3)
    x = vectors((40, 4, 128), ms.BF16, 5)
    pos = torch.arange(40, dtype=torch.int32, device="cuda")[None]
    ko, vo = (torch.zeros((40, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ms.kv_cache_write(kd, 1, x[:, :2], x[:, 2:], pos, c, ws, stream=s)
    ms.kv_cache_read(kd, 1, pos, c, ko, vo, ws, stream=s)
    s.synchronize()
    assert torch.equal(ko, x[:, :2]) and torch.equal(vo, x[:, 2:])
