"""Refusals of the planning, rotary and delta-rule calls (CPU): every bad argument is answered by its documented code
before anything is launched, at the C entries and in the binding."""
import copy
import ctypes
import os
import pickle

import pytest
import torch

import moe_expert_step_gb300 as ms

FAKE = 1 << 20          # an aligned, never-dereferenced address
KV = dict(Hq=16, Hkv=2, D=128, page=64, n_pages=100, max_pages=8, dtype=ms.BF16)
DD = dict(Hk=2, Hv=4, Dk=128, Dv=64, n_slots=5, dtype=ms.BF16)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(ms.library_path()):
        ms.build()
    return ms.lib()


# ------------------------------------------------------------------------------ kv_cache_plan


def plan(L, dims=None, **kw):
    a = dict(R=3, n=32, kv_len=FAKE, n_new=FAKE, ring=FAKE, head=FAKE, head_out=FAKE, table=FAKE, new_len=FAKE + 64, pos=FAKE,
             slots=None, ws=FAKE, bytes=512) | kw
    kd = ms.KvDims(**{**KV, **(dims or {})})
    return L.kv_cache_plan(kd._c, a["R"], a["n"], a["kv_len"], a["n_new"], a["ring"], a["head"], a["head_out"], a["table"],
                           a["new_len"], a["pos"], a["slots"], a["ws"], a["bytes"], None)


def test_plan_arguments(L):
    for kw in (dict(R=0), dict(n=0), dict(n=-1), dict(kv_len=None), dict(n_new=None), dict(ring=None), dict(head=None),
               dict(head_out=None), dict(table=None), dict(new_len=None), dict(pos=None), dict(new_len=FAKE),
               dict(n_new=FAKE + 64), dict(dims=dict(page=0))):
        assert plan(L, **kw) == ms.EINVAL, kw
    for name in ("kv_len", "n_new", "ring", "head", "head_out", "table", "new_len", "pos", "slots"):
        assert plan(L, **{name: FAKE + 130}) == ms.EALIGN, name
    for kw in (dict(ws=None), dict(ws=FAKE + 128), dict(bytes=511)):
        assert plan(L, **kw) == ms.EWORKSPACE, kw
    for kw in (dict(R=(1 << 20) + 1), dict(dims=dict(D=96)), dict(dims=dict(page=48))):
        assert plan(L, **kw) == ms.EUNSUPPORTED, kw


def test_plan_binding(L):
    kd = ms.KvDims(**KV)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    good = dict(kv_len=i32(3), n_new=i32(3), ring=i32(100), head=i32(2), head_out=i32(2), table=i32(3, 8), new_len=i32(3),
                pos=i32(3, 32), ws=torch.zeros(512, dtype=torch.uint8))

    def refused(match, **kw):
        a = good | kw
        with pytest.raises(ms.MoeStepError, match=match) as e:
            ms.kv_cache_plan(kd, 3, a["kv_len"], a["n_new"], a["ring"], a["head"], a["head_out"], a["table"], a["new_len"],
                             a["pos"], a["ws"], slots=a.get("slots"))
        assert e.value.code == ms.EINVAL

    refused("kv_len must be contiguous", kv_len=i32(4))
    refused("kv_len must be contiguous", kv_len=torch.zeros(3, dtype=torch.int64))
    refused("kv_len must be on the GPU")


@pytest.mark.gpu
def test_plan_binding_on_the_gpu():
    kd = ms.KvDims(**KV)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    good = dict(kv_len=i32(3), n_new=i32(3), ring=i32(100), head=i32(2), head_out=i32(2), table=i32(3, 8), new_len=i32(3),
                pos=i32(3, 32), slots=None, ws=ms.kv_workspace(kd, 3, 1))

    def call(**kw):
        a = good | kw
        ms.kv_cache_plan(kd, 3, a["kv_len"], a["n_new"], a["ring"], a["head"], a["head_out"], a["table"], a["new_len"],
                         a["pos"], a["ws"], slots=a["slots"])

    call()
    call(slots=i32(3, 32), table=i32(5, 8))
    for name, bad in (("n_new", i32(3, 1)), ("ring", i32(99)), ("head", i32(3)), ("head_out", i32(1)), ("table", i32(2, 8)),
                      ("table", i32(3, 9)), ("new_len", i32(2)), ("pos", i32(2, 32)), ("pos", i32(32, 3).t()),
                      ("slots", i32(3, 31)), ("slots", torch.zeros((3, 32), device="cuda"))):
        with pytest.raises(ms.MoeStepError, match=name):
            call(**{name: bad})
    with pytest.raises(ms.MoeStepError, match="bytes on the GPU"):
        call(ws=torch.zeros(512, dtype=torch.uint8))
    with pytest.raises(ms.MoeStepError):  # new_len may not be kv_len
        call(new_len=good["kv_len"])
    torch.cuda.synchronize()


# ------------------------------------------------------------------------------ rotary positions


def rotary(L, dims=None, **kw):
    a = dict(R=2, n=3, q=FAKE, q_ld=16 * 128, k=FAKE, k_ld=2 * 128, pos=FAKE, freq=FAKE, rot=64, pairs=0, mscale=1.0, qo=FAKE * 2,
             qo_ld=16 * 128, ko=FAKE * 3, ko_ld=2 * 128) | kw
    kd = ms.KvDims(**{**KV, **(dims or {})})
    return L.block_rotary(kd._c, a["R"], a["n"], a["q"], a["q_ld"], a["k"], a["k_ld"], a["pos"], a["freq"], a["rot"], a["pairs"],
                          a["mscale"], a["qo"], a["qo_ld"], a["ko"], a["ko_ld"], None)


def test_rotary_arguments(L):
    for kw in (dict(R=0), dict(n=0), dict(pos=None), dict(freq=None), dict(rot=0), dict(rot=63), dict(rot=-2), dict(rot=130),
               dict(mscale=float("nan")), dict(mscale=float("inf")), dict(q=None), dict(qo=None), dict(k=None), dict(ko=None),
               dict(q=None, qo=None, k=None, ko=None), dict(q_ld=16 * 128 - 1), dict(k_ld=2 * 128 - 1), dict(qo_ld=100),
               dict(ko_ld=0), dict(qo=FAKE, qo_ld=16 * 128 + 8), dict(ko=FAKE, ko_ld=2 * 128 + 8), dict(dims=dict(Hq=0))):
        assert rotary(L, **kw) == ms.EINVAL, kw
    for kw in (dict(q=FAKE + 1), dict(ko=FAKE + 1), dict(pos=FAKE + 2), dict(freq=FAKE + 4), dict(q=FAKE + 2, dims=dict(dtype=ms.F32))):
        assert rotary(L, **kw) == ms.EALIGN, kw
    for kw in (dict(R=1 << 30, n=1 << 30), dict(dims=dict(D=96), rot=32)):
        assert rotary(L, **kw) == ms.EUNSUPPORTED, kw


@pytest.mark.parametrize("bad", [
    dict(rot=0), dict(rot=7), dict(rot=-4), dict(base=1.0), dict(base=float("inf")), dict(base=float("nan")), dict(scaling=-1),
    dict(scaling=4), dict(factor=0.0), dict(factor=float("nan")), dict(original=0.0), dict(low=0.0), dict(low=4.0),
    dict(high=float("inf")), dict(freq=None)])
def test_frequency_arguments(L, bad):
    a = dict(rot=64, base=1e4, scaling=ms.ROTARY_ROTATIONS, factor=4.0, original=4096.0, low=1.0, high=4.0, freq=FAKE) | bad
    call = lambda **kw: L.rotary_frequencies(*(a | kw).values(), None)  # noqa: E731
    assert call() == ms.EINVAL
    assert call(**dict(rot=64, base=1e4, scaling=0, factor=4.0, original=4096.0, low=1.0, high=4.0, freq=FAKE + 4)) == ms.EALIGN
    assert call(**dict(rot=4098, base=1e4, scaling=0, factor=0.0, original=0.0, low=0.0, high=0.0, freq=FAKE)) == ms.EUNSUPPORTED


def test_rotary_binding(L):
    kd = ms.KvDims(**KV)
    bf = torch.bfloat16
    q, k = torch.zeros(6, 16, 128, dtype=bf), torch.zeros(6, 2, 128, dtype=bf)
    pos, freq = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(32, dtype=torch.int64)

    def refused(match, *a):
        with pytest.raises(ms.MoeStepError, match=match) as e:
            ms.block_rotary(kd, *a)
        assert e.value.code == ms.EINVAL

    refused("pos must be .R, n", q, k, pos.view(-1), freq, q, k)
    refused("pos must be contiguous", q, k, pos.float(), freq, q, k)
    refused("pos must be on the GPU", q, k, pos, freq, q, k)
    with pytest.raises(ms.MoeStepError, match="rot must be even"):
        ms.rotary_frequencies(7, 1e4)


@pytest.mark.gpu
def test_rotary_binding_on_the_gpu():
    kd = ms.KvDims(**KV)
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    pos, freq = torch.zeros((2, 3), dtype=torch.int32, device="cuda"), ms.rotary_frequencies(64, 1e4)
    q, k = z(6, 16, 128), z(6, 2, 128)
    ms.block_rotary(kd, q, k, pos, freq, z(6, 16, 128), z(6, 2, 128))
    ms.block_rotary(kd, None, k, pos, freq, None, k)
    for bad in (z(5, 16, 128), z(6, 15, 128), z(6, 16, 64), z(6, 16, 128).float(), z(6, 16, 256)[:, :, ::2], z(6, 128, 16).transpose(1, 2),
                torch.zeros(6, 16, 128, dtype=torch.bfloat16)):
        for a in ((bad, k, pos, freq, q, k), (q, k, pos, freq, bad, k)):
            with pytest.raises(ms.MoeStepError, match="q"):
                ms.block_rotary(kd, *a)
    for a in ((q, None, pos, freq, None, None), (q, k, pos, freq, q, None), (q, None, pos, freq, q, k), (None, k, pos, freq, q, k), (q, k, pos, ms.rotary_frequencies(130, 1e4), q, k),
              (q, k, pos, freq.float(), q, k)):
        with pytest.raises(ms.MoeStepError):
            ms.block_rotary(kd, *a)
    torch.cuda.synchronize()


# ------------------------------------------------------------------------------ the delta rule


BAD_DELTA = [
    (dict(Hk=0), ms.EINVAL), (dict(Hv=0), ms.EINVAL), (dict(Dk=0), ms.EINVAL), (dict(Dv=-1), ms.EINVAL), (dict(n_slots=0), ms.EINVAL),
    (dict(dtype=ms.FP8), ms.EINVAL), (dict(dtype=9), ms.EINVAL), (dict(Hv=5), ms.EUNSUPPORTED), (dict(Hv=2048), ms.EUNSUPPORTED),
    (dict(Dk=96), ms.EUNSUPPORTED), (dict(Dk=256), ms.EUNSUPPORTED), (dict(Dv=32), ms.EUNSUPPORTED),
]


def delta(L, dims=None, **kw):
    a = dict(R=2, n=4, q=FAKE, q_ld=2 * 128, k=FAKE, k_ld=2 * 128, v=FAKE, v_ld=4 * 64, g=FAKE, beta=FAKE, length=None, slot=None,
             fresh=None, state=FAKE, state_out=None, scale=1.0, eps=0.0, out=FAKE, ws=FAKE, bytes=1 << 40) | kw
    dd = ms.DeltaDims(**{**DD, **(dims or {})})
    return L.block_delta_rule(dd._c, a["R"], a["n"], a["q"], a["q_ld"], a["k"], a["k_ld"], a["v"], a["v_ld"], a["g"], a["beta"],
                              a["length"], a["slot"], a["fresh"], a["state"], a["state_out"], a["scale"], a["eps"], a["out"],
                              a["ws"], a["bytes"], None)


@pytest.mark.parametrize("bad,code", BAD_DELTA)
def test_delta_dims(L, bad, code):
    n = ctypes.c_size_t(0)
    assert L.moestep_delta_workspace_size(ms.DeltaDims(**{**DD, **bad})._c, 1, 1, ctypes.byref(n)) == code
    assert delta(L, dims=bad, v_ld=1 << 20) == code


def test_delta_workspace_size(L):
    dd = ms.DeltaDims(**DD)
    assert L.moestep_delta_workspace_size(dd._c, 1, 1, None) == ms.EINVAL
    n = ctypes.c_size_t(0)
    for R, m, code in ((0, 1, ms.EINVAL), (1, 0, ms.EINVAL), (1 << 23, 1, ms.EUNSUPPORTED), (1, (1 << 30) + 1, ms.EUNSUPPORTED),
                       (1 << 16, 1 << 16, ms.EUNSUPPORTED)):
        assert L.moestep_delta_workspace_size(dd._c, R, m, ctypes.byref(n)) == code, (R, m)
    assert ms.delta_workspace_size(dd, 1, 1) == 512
    one, two = ms.delta_workspace_size(dd, 1, 4096), ms.delta_workspace_size(dd, 2, 4096)
    assert 512 < one < two
    assert ms.delta_workspace_size(ms.DeltaDims(**{**DD, "dtype": ms.F32}), 2, 4096) == 512


def test_delta_arguments(L):
    for kw in (dict(R=0), dict(n=0), dict(q=None), dict(k=None), dict(v=None), dict(g=None), dict(beta=None), dict(state=None),
               dict(out=None), dict(q_ld=255), dict(k_ld=248), dict(v_ld=0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(eps=-1e-6), dict(eps=float("nan")), dict(R=6)):  # six requests, five slots, no slot numbers
        assert delta(L, **kw) == ms.EINVAL, kw
    for kw in (dict(q=FAKE + 8), dict(k=FAKE + 2), dict(v=FAKE + 8), dict(q_ld=257), dict(state=FAKE + 8), dict(state_out=FAKE + 4),
               dict(out=FAKE + 8), dict(g=FAKE + 2), dict(beta=FAKE + 1), dict(length=FAKE + 2), dict(slot=FAKE + 1)):
        assert delta(L, **kw) == ms.EALIGN, kw
    need = ms.delta_workspace_size(ms.DeltaDims(**DD), 2, 100)
    for kw in (dict(ws=None), dict(ws=FAKE + 128), dict(bytes=511), dict(n=100, bytes=need - 1)):
        assert delta(L, **kw) == ms.EWORKSPACE, kw


def delta_tensors(device, R=2, n=3, dtype=torch.bfloat16):
    T = R * n
    z = lambda *s, t=dtype: torch.zeros(s, dtype=t, device=device)  # noqa: E731
    f = torch.float32
    return dict(q=z(T, 2, 128), k=z(T, 2, 128), v=z(T, 4, 64), g=z(T, 4, t=f), beta=z(T, 4, t=f), state=z(5, 4, 64, 128, t=f),
                out=z(T, 4, 64), ws=torch.zeros(512, dtype=torch.uint8, device=device))


def test_delta_binding(L):
    dd = ms.DeltaDims(**DD)
    good = delta_tensors("cpu")

    def refused(match, R=2, **kw):
        a = good | kw
        with pytest.raises(ms.MoeStepError, match=match) as e:
            ms.block_delta_rule(dd, R, a["q"], a["k"], a["v"], a["g"], a["beta"], a["state"], a["out"], a["ws"])
        assert e.value.code == ms.EINVAL

    refused("q must be")  # on the GPU
    refused("R . n rows", R=4)
    refused("R . n rows", R=0)


@pytest.mark.gpu
def test_delta_binding_on_the_gpu():
    dd = ms.DeltaDims(**DD)
    good = delta_tensors("cuda")
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8

    def call(**kw):
        a = good | kw
        ms.block_delta_rule(dd, 2, a["q"], a["k"], a["v"], a["g"], a["beta"], a["state"], a["out"], a["ws"],
                            **{k: a[k] for k in ("state_out", "slot", "length", "fresh") if k in a})

    call()
    call(state_out=z(5, 4, 64, 128, t=f32), slot=z(2, t=i32) + torch.arange(2, device="cuda", dtype=i32), length=z(2, t=i32),
         fresh=z(2, t=u8))
    for name, bads in dict(
            q=(z(6, 2, 64), z(6, 3, 128), z(6, 2, 128, t=f32), z(6, 2, 256)[:, :, ::2]), k=(z(5, 2, 128), z(6, 2, 128).cpu()),
            v=(z(6, 4, 128), z(6, 2, 64)), g=(z(6, 4), z(6, 3, t=f32), z(4, 6, t=f32).t()), beta=(z(6, 4, t=torch.float16),),
            state=(z(4, 4, 64, 128, t=f32), z(5, 4, 128, 64, t=f32), z(5, 4, 64, 128)), out=(z(6, 4, 64, t=f32), z(6, 4, 128)[:, :, ::2]),
            state_out=(z(4, 4, 64, 128, t=f32),), slot=(z(3, t=i32), z(2, t=torch.int64)), length=(z(2, 1, t=i32),),
            fresh=(z(2, t=torch.bool), z(2, t=i32))).items():
        for bad in bads:
            with pytest.raises(ms.MoeStepError, match="block_delta_rule: " + name):
                call(**{name: bad})
    with pytest.raises(ms.MoeStepError, match="bytes on the GPU"):
        call(ws=good["ws"].cpu())
    torch.cuda.synchronize()


def test_dims_can_be_copied():
    dd = ms.DeltaDims(**DD)
    for other in (copy.deepcopy(dd), pickle.loads(pickle.dumps(dd))):
        assert other == dd and other is not dd and other._c is not dd._c
