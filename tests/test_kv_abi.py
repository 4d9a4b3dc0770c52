"""Refusals of the cache, attention and residual-norm calls (CPU): every bad argument is answered
by its documented code before anything is launched, at the C entries and in the binding."""
import ctypes

import pytest
import torch

import moe_expert_step_gb300 as ms

FAKE = 1 << 20          # an aligned, never-dereferenced address
GOOD = dict(Hq=16, Hkv=2, D=128, page=64, n_pages=100, max_pages=8, dtype=ms.BF16)


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(ms.library_path()):
        ms.build()
    return ms.lib()


def cache(dtype=ms.BF16, **kw):
    e = FAKE if dtype == ms.FP8 else None
    f = dict(k=FAKE, v=FAKE, k_exp=e, v_exp=e, table=FAKE) | kw
    return ms.KvCache(f["k"], f["v"], f["k_exp"], f["v_exp"], f["table"])


BAD_DIMS = [
    (dict(Hq=0), ms.EINVAL), (dict(Hkv=0), ms.EINVAL), (dict(D=0), ms.EINVAL), (dict(page=0), ms.EINVAL),
    (dict(n_pages=0), ms.EINVAL), (dict(max_pages=-1), ms.EINVAL), (dict(dtype=3), ms.EINVAL),
    (dict(Hq=15), ms.EUNSUPPORTED), (dict(Hq=2048), ms.EUNSUPPORTED), (dict(D=96), ms.EUNSUPPORTED),
    (dict(page=48), ms.EUNSUPPORTED), (dict(page=256), ms.EUNSUPPORTED),
    (dict(n_pages=1 << 30), ms.EUNSUPPORTED), (dict(max_pages=1 << 25), ms.EUNSUPPORTED),
]


@pytest.mark.parametrize("bad,code", BAD_DIMS)
def test_bad_dims(L, bad, code):
    kd = ms.KvDims(**{**GOOD, **bad})
    n = ctypes.c_size_t(0)
    assert L.moestep_kv_workspace_size(kd._c, 1, 1, ctypes.byref(n)) == code
    c = cache()
    assert L.kv_cache_write(kd._c, 1, 1, FAKE, FAKE, 1 << 20, FAKE, c, FAKE, 512, None) == code
    assert L.kv_cache_read(kd._c, 1, 1, FAKE, c, FAKE, FAKE, FAKE, 512, None) == code
    assert L.block_attention(kd._c, 1, 1, FAKE, 1 << 20, FAKE, c, 1.0, 0, 0, FAKE, None, FAKE, 1 << 40, None) == code


@pytest.mark.parametrize("R,n_q,code", [(0, 1, ms.EINVAL), (1, 0, ms.EINVAL), (1, 1025, ms.EUNSUPPORTED),
                                        (1 << 21, 1, ms.EUNSUPPORTED)])
def test_bad_counts(L, R, n_q, code):
    kd = ms.KvDims(**GOOD)
    n = ctypes.c_size_t(0)
    assert L.moestep_kv_workspace_size(kd._c, R, n_q, ctypes.byref(n)) == code
    assert L.moestep_kv_workspace_size(kd._c, 1, 1, None) == ms.EINVAL


@pytest.mark.parametrize("dtype", [ms.BF16, ms.F32, ms.FP8])
def test_attention_arguments(L, dtype):
    kd = ms.KvDims(**{**GOOD, "dtype": dtype})
    n = ms.kv_workspace_size(kd, 2, 4)
    ok = dict(q=FAKE, ld=16 * 128, len=FAKE, cache=cache(dtype), scale=0.1, window=0, out=FAKE, ws=FAKE, n=n)

    def call(**kw):
        a = ok | kw
        return L.block_attention(kd._c, 2, 4, a["q"], a["ld"], a["len"], a["cache"], a["scale"], 0, a["window"],
                                 a["out"], None, a["ws"], a["n"], None)

    for kw in (dict(q=None), dict(len=None), dict(out=None), dict(cache=None), dict(cache=cache(dtype, k=None)),
               dict(cache=cache(dtype, v=None)), dict(cache=cache(dtype, table=None)), dict(ld=16 * 128 - 8),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(window=-1)):
        assert call(**kw) == ms.EINVAL, kw
    if dtype == ms.FP8:
        assert call(cache=cache(dtype, k_exp=None)) == ms.EINVAL
        assert call(cache=cache(dtype, v_exp=FAKE + 8)) == ms.EALIGN
    for kw in (dict(q=FAKE + 8), dict(out=FAKE + 4), dict(ld=16 * 128 + 2), dict(cache=cache(dtype, k=FAKE + 8)),
               dict(cache=cache(dtype, table=FAKE + 4))):
        assert call(**kw) == ms.EALIGN, kw
    for kw in (dict(ws=None), dict(ws=FAKE + 128), dict(n=n - 1)):
        assert call(**kw) == ms.EWORKSPACE, kw


def test_copy_arguments(L):
    kd = ms.KvDims(**GOOD)
    c = cache()
    w = lambda k=FAKE, v=FAKE, ld=256, pos=FAKE, c=c, ws=FAKE, n=512, R=1, m=4: L.kv_cache_write(  # noqa: E731
        kd._c, R, m, k, v, ld, pos, c, ws, n, None)
    for kw in (dict(k=None), dict(v=None), dict(pos=None), dict(c=None), dict(ld=255), dict(R=0), dict(m=0)):
        assert w(**kw) == ms.EINVAL, kw
    for kw in (dict(k=FAKE + 2), dict(v=FAKE + 8), dict(ld=260), dict(c=cache(v=FAKE + 4))):
        assert w(**kw) == ms.EALIGN, kw
    for kw in (dict(ws=None), dict(ws=FAKE + 64), dict(n=511)):
        assert w(**kw) == ms.EWORKSPACE, kw
    assert w(R=1 << 16, m=1 << 16) == ms.EUNSUPPORTED
    r = lambda k=FAKE, v=FAKE, pos=FAKE: L.kv_cache_read(kd._c, 1, 4, pos, c, k, v, FAKE, 512, None)  # noqa: E731
    assert r(k=None) == r(v=None) == r(pos=None) == ms.EINVAL
    assert r(k=FAKE + 4) == r(v=FAKE + 8) == ms.EALIGN


def test_residual_norm_arguments(L):
    d = ms.ModelDims(H=2048, E=256, k=8, I=512, Is=512, V=152064, P=32, dtype=ms.BF16).c()
    ok = dict(T=4, y=FAKE, yt=ms.BF16, wp=FAKE, g=FAKE, ld=2048, s=1.0, h=FAKE, o=FAKE, wq=FAKE, x=FAKE, eps=1e-6)

    def call(**kw):
        a = ok | kw
        return L.block_residual_norm(ctypes.byref(d), a["T"], a["y"], a["yt"], a["wp"], a["g"], a["ld"], a["s"],
                                     a["h"], a["o"], a["wq"], a["x"], a["eps"], None)

    for kw in (dict(T=0), dict(y=None), dict(h=None), dict(o=None), dict(yt=ms.FP8), dict(yt=9), dict(eps=0.0),
               dict(eps=-1e-6), dict(eps=float("nan")), dict(s=float("inf")), dict(ld=-4), dict(ld=1024)):
        assert call(**kw) == ms.EINVAL, kw
    for kw in (dict(y=FAKE + 8), dict(wp=FAKE + 2), dict(g=FAKE + 4), dict(h=FAKE + 8), dict(o=FAKE + 8),
               dict(wq=FAKE + 2), dict(x=FAKE + 8), dict(ld=2050)):
        assert call(**kw) == ms.EALIGN, kw
    bad = ms.ModelDims(H=2000, E=256, k=8, I=512, Is=512, V=1, P=32, dtype=ms.BF16).c()
    assert L.block_residual_norm(ctypes.byref(bad), 4, FAKE, ms.BF16, None, None, 0, 1.0, FAKE, FAKE, None, FAKE, 1e-6,
                                 None) == ms.EUNSUPPORTED


def test_binding_refuses_shapes(L):
    kd = ms.KvDims(**GOOD)
    bf, i32 = torch.bfloat16, torch.int32
    c = cache()
    ws = torch.zeros(512, dtype=torch.uint8)

    def refused(match, f, *a, **k):
        with pytest.raises(ms.MoeStepError, match=match) as e:
            f(*a, **k)
        assert e.value.code == ms.EINVAL

    q, out, n = torch.zeros(4, 16, 128, dtype=bf), torch.zeros(4, 16, 128, dtype=bf), torch.zeros(2, dtype=i32)
    refused("q must be .tokens", ms.block_attention, kd, 2, q.float(), n, c, out, ws, 1.0)
    refused("q must be .tokens", ms.block_attention, kd, 2, q[:, :8], n, c, out, ws, 1.0)
    refused("q must be .tokens", ms.block_attention, kd, 2, torch.zeros(4, 16, 256, dtype=bf)[:, :, ::2], n, c, out, ws, 1.0)
    refused("q must be on the GPU", ms.block_attention, kd, 2, q, n, c, out, ws, 1.0)
    refused("contiguous", ms.kv_cache, torch.zeros(4, 4).t(), q, n)
    kv = torch.zeros(6, 4, 128, dtype=bf)
    refused("pos must be contiguous", ms.kv_cache_write, kd, 2, kv[:, :2], kv[:, 2:], torch.zeros(3, 2, dtype=i32).t(), c, ws)
    refused("pos must be contiguous", ms.kv_cache_write, kd, 2, kv[:, :2], kv[:, 2:],
            torch.zeros(2, 3, dtype=torch.int64), c, ws)
    d = ms.ModelDims(H=2048, E=256, k=8, I=512, Is=512, V=152064)
    y, h = torch.zeros(3, 2048), torch.zeros(3, 1024)
    refused("y must be", ms.block_residual_norm, d, y.double(), y, y, None)
    refused("y must be contiguous", ms.block_residual_norm, d, h, h, h, None)


@pytest.mark.parametrize("what,dtype", [("q", torch.float16), ("q", torch.int16), ("out", torch.float16),
                                        ("kv_len", torch.float32), ("lse", torch.int32)])
def test_binding_refuses_types_of_the_right_size(L, what, dtype):
    kd = ms.KvDims(**GOOD)
    t = dict(q=torch.zeros(4, 16, 128, dtype=torch.bfloat16), kv_len=torch.zeros(4, dtype=torch.int32),
             out=torch.zeros(4, 16, 128, dtype=torch.bfloat16), lse=torch.zeros(4, 16))
    t[what] = t[what].to(dtype)
    with pytest.raises(ms.MoeStepError) as e:
        ms.block_attention(kd, 4, t["q"], t["kv_len"], cache(), t["out"], torch.zeros(512, dtype=torch.uint8), 1.0,
                           lse=t["lse"])
    assert e.value.code == ms.EINVAL


def test_binding_refuses_other_types_in_the_norm(L):
    d = ms.ModelDims(H=256, E=8, k=2, I=64, Is=64, V=128)
    h = torch.zeros(2, 256)
    for y, x in ((h.half(), None), (h, h.half()), (h, h)):
        with pytest.raises(ms.MoeStepError) as e:
            ms.block_residual_norm(d, y, h, h, x)
        assert e.value.code == ms.EINVAL


def test_dims_can_be_copied():
    import copy
    import pickle
    kd = ms.KvDims(**GOOD)
    for other in (copy.deepcopy(kd), pickle.loads(pickle.dumps(kd))):
        assert other == kd and other is not kd and other._c is not kd._c
