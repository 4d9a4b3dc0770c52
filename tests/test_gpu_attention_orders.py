"""block_attention in the orders of segments, row tiles and windows that its division of the work can
bring, against the float64 oracle with the bounds of test_gpu_attention.py."""
import pytest
import torch

import moe_expert_step_gb300 as ms
from tests.test_gpu_attention import Setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n_q", [4, 8, 16])
@pytest.mark.parametrize("dtype", [ms.BF16, ms.FP8])
def test_segments_that_one_stream_has_no_tile_of(dtype, n_q, D):
    """Row tiles of 32, 64 and 128; every CTA goes through three segments of one key tile, which the
    second stream only passes."""
    s = Setup(dtype, [1 + (7 * r) % 12 for r in range(57)], n_q, Hkv=8, G=8, D=D, page=16, seed=21)
    out, ls = s.run()
    s.check(out, ls)
    for _ in range(20):
        o2, l2 = s.run()
        assert torch.equal(o2, out) and torch.equal(l2, ls)


@pytest.mark.parametrize("dtype", [ms.BF16, ms.F32, ms.FP8])
def test_windows_about_as_long_as_32_bits(dtype):
    """A window longer than the request hides nothing, up to the longest that the longest page table allows and
    beyond it."""
    n_q, max_pages = 512, (1 << 27) - 16
    s = Setup(dtype, [600], n_q, 1, 1, 64, 16, seed=22)
    table = torch.empty((1, max_pages), dtype=torch.int32, device="cuda")
    table[:, :s.table.shape[1]] = s.table
    s.kd = ms.KvDims(Hq=1, Hkv=1, D=64, page=16, n_pages=s.kd.n_pages, max_pages=max_pages, dtype=dtype)
    s.cache = ms.kv_cache(*s.pools, table, *s.cache._tensors[3:])
    for n in (600, 10):
        s.len.fill_(n)
        s.window = 0
        want = s.run(True)
        for s.window in (1 << 30, 2 ** 31 - 1 - n_q, 16 * max_pages, 2 ** 31 - 1, 2 ** 31, 2 ** 40):
            out, ls = s.run(True)
            assert torch.equal(out, want[0]) and torch.equal(ls, want[1]), (n, s.window)
        for s.window in (2 ** 31 - n_q, 16 * max_pages - 1):  # shorter than the table's positions
            with pytest.raises(ms.MoeStepError) as e:
                s.run(True)
            assert e.value.code == ms.EUNSUPPORTED
    assert ms.read_device_error(s.ws) == ms.OK


@pytest.mark.parametrize("dtype", [ms.BF16, ms.F32, ms.FP8])
def test_one_row_has_no_stride(dtype):
    """A single token's keys, values and queries are taken from rows of different and odd widths."""
    kd = ms.KvDims(Hq=4, Hkv=2, D=64, page=16, n_pages=1, max_pages=1, dtype=dtype)
    act = torch.float32 if dtype == ms.F32 else torch.bfloat16
    store = {ms.BF16: torch.bfloat16, ms.F32: torch.float32, ms.FP8: torch.float8_e4m3fn}[dtype]
    results = []
    for k_ld, v_ld, q_ld in ((128, 128, 256), (1024, 128, 259), (131, 2000, 777), (1, 1, 1)):
        pools = [torch.zeros((1, 2, 16, 64), device="cuda").to(store) for _ in "kv"]
        exps = [torch.zeros((1, 2, 16), dtype=torch.uint8, device="cuda") if dtype == ms.FP8 else None for _ in "kv"]
        cache = ms.kv_cache(*pools, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), *exps)
        ws = ms.kv_workspace(kd, 1, 1)
        g = torch.Generator(device="cuda").manual_seed(1)
        new = lambda h, ld: torch.randn(h * 64, generator=g, device="cuda").to(act).as_strided((1, h, 64), (ld, 64, 1))  # noqa: E731
        k, v, q, out = new(2, k_ld), new(2, v_ld), new(4, q_ld), torch.empty((1, 4, 64), dtype=act, device="cuda")
        ms.kv_cache_write(kd, 1, k, v, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), cache, ws)
        ms.block_attention(kd, 1, q, torch.ones(1, dtype=torch.int32, device="cuda"), cache, out, ws, 0.1)
        assert ms.read_device_error(ws) == ms.OK
        results.append((pools[0].float(), pools[1].float(), out))
    for r in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, results[0]))
    assert torch.equal(results[0][2][0, :2], results[0][2][0, 1:2].expand(2, 64))  # one key: its value


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("window", [1, 40, 70, 128, 300])
@pytest.mark.parametrize("n_q,D", [(20, 64), (20, 128), (50, 64), (50, 128), (80, 64), (80, 128), (150, 128), (200, 64)])
@pytest.mark.parametrize("dtype", [ms.BF16, ms.F32, ms.FP8])
def test_windows_over_every_row_tile(dtype, n_q, D, window, causal):
    """Row tiles of 64, 128 and 256 and two of 256; windows that begin in either half of a key tile."""
    s = Setup(dtype, [400, 17, 0, 139], n_q, 1, 2, D, 32, window=window, seed=23)
    s.check(*s.run(causal), causal)


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 128), (False, 50)])
@pytest.mark.parametrize("lengths,n_q,G,D", [([700, 130], 130, 4, 128), ([515, 1, 300], 260, 2, 128), ([1024], 1024, 1, 128),
                                             ([1500], 1024, 2, 64), ([777], 513, 3, 128)])
@pytest.mark.parametrize("dtype", [ms.BF16, ms.F32, ms.FP8])
def test_prompts(dtype, lengths, n_q, G, D, causal, window):
    """Up to 1024 new tokens and eight row tiles, whole and shared by CTAs."""
    s = Setup(dtype, lengths, n_q, 1, G, D, 64, window=window, seed=24)
    out, ls = s.run(causal)
    s.check(out, ls, causal)
    o2, l2 = s.run(causal)
    assert torch.equal(out, o2) and torch.equal(ls, l2)
