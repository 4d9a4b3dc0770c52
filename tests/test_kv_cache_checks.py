"""What the binding refuses of a cache: tensors that are not one, and one that is not the call's.  Each
refusal is named by its message, and the unmodified arguments are accepted."""
import pytest
import torch

import moe_expert_step_gb300 as ms

N, HKV, PAGE, D, R, MAX = 6, 2, 16, 64, 3, 4
STORE = {ms.BF16: torch.bfloat16, ms.F32: torch.float32, ms.FP8: torch.float8_e4m3fn}


def tensors(dtype=ms.BF16, device="cpu", n=N, hkv=HKV, page=PAGE, d=D, rows=R, width=MAX, table=torch.int32):
    pool = lambda: torch.zeros((n, hkv, page, d), dtype=torch.uint8 if dtype == ms.FP8 else STORE[dtype],  # noqa: E731
                               device=device)
    exp = lambda: torch.zeros((n, hkv, page), dtype=torch.uint8, device=device) if dtype == ms.FP8 else None  # noqa: E731
    return dict(k=pool(), v=pool(), table=torch.zeros((rows, width), dtype=table, device=device), k_exp=exp(), v_exp=exp())


BAD = [
    (ms.BF16, dict(table=torch.zeros((R, MAX), dtype=torch.int64)), "table must be"),
    (ms.BF16, dict(table=torch.zeros(R * MAX, dtype=torch.int32)), "table must be"),
    (ms.BF16, dict(v=torch.zeros((N, HKV, PAGE, D))), "k and v must be"),
    (ms.BF16, dict(v=torch.zeros((N, HKV, PAGE, D + 64), dtype=torch.bfloat16)), "k and v must be"),
    (ms.BF16, dict(k=torch.zeros((N, HKV, PAGE, D), dtype=torch.float16)), "k and v must be"),
    (ms.F32, dict(k=torch.zeros((N, HKV, PAGE * D)), v=torch.zeros((N, HKV, PAGE * D))), "k and v must be"),
    (ms.FP8, dict(k_exp=None), "k_exp and v_exp must be"),
    (ms.FP8, dict(v_exp=torch.zeros((N, HKV, PAGE + 1), dtype=torch.uint8)), "k_exp and v_exp must be"),
    (ms.FP8, dict(v_exp=torch.zeros((N, HKV, PAGE), dtype=torch.int32)), "k_exp and v_exp must be"),
    (ms.BF16, dict(k=torch.zeros((N, HKV, D, PAGE), dtype=torch.bfloat16).transpose(2, 3)), "contiguous"),
    (ms.BF16, {}, "must be on the GPU"),
    (ms.FP8, {}, "must be on the GPU"),
]


@pytest.mark.parametrize("dtype,bad,match", BAD)
def test_what_is_no_cache(dtype, bad, match):
    with pytest.raises(ms.MoeStepError, match=match) as e:
        ms.kv_cache(**(tensors(dtype) | bad))
    assert e.value.code == ms.EINVAL


class Calls:
    """The three calls with arguments that fit a cache of the given tensors."""

    def __init__(self, dtype, **kw):
        self.kd = ms.KvDims(Hq=2 * HKV, Hkv=HKV, D=D, page=PAGE, n_pages=N, max_pages=MAX, dtype=dtype)
        self.cache = ms.kv_cache(**tensors(dtype, "cuda", **kw))
        self.ws = ms.kv_workspace(self.kd, R, 1)
        act = torch.float32 if dtype == ms.F32 else torch.bfloat16
        z = lambda h: torch.zeros((R, h, D), dtype=act, device="cuda")  # noqa: E731
        self.k, self.v, self.q, self.out = z(HKV), z(HKV), z(2 * HKV), z(2 * HKV)
        self.n = torch.ones(R, dtype=torch.int32, device="cuda")
        self.lse = torch.zeros((R, 2 * HKV), device="cuda")
        self.pos = torch.full((R, 1), -1, dtype=torch.int32, device="cuda")

    def all(self, kd=None, ws=None):
        kd, ws = kd or self.kd, self.ws if ws is None else ws
        return [lambda: ms.kv_cache_write(kd, R, self.k, self.v, self.pos, self.cache, ws),
                lambda: ms.kv_cache_read(kd, R, self.pos, self.cache, self.k, self.v, ws),
                lambda: ms.block_attention(kd, R, self.q, self.n, self.cache, self.out, ws, 0.1, lse=self.lse)]


def refused(calls, match):
    for call in calls:
        with pytest.raises(ms.MoeStepError, match=match) as e:
            call()
        assert e.value.code == ms.EINVAL


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [ms.BF16, ms.F32, ms.FP8])
def test_a_cache_that_is_not_the_calls(dtype):
    for kw in (dict(n=N - 1), dict(hkv=HKV + 1), dict(page=2 * PAGE), dict(d=2 * D), dict(rows=R - 1),
               dict(width=MAX + 1), dict(width=MAX - 1)):
        refused(Calls(dtype, **kw).all(), "the cache does not have")
    other = {ms.BF16: ms.FP8, ms.F32: ms.BF16, ms.FP8: ms.BF16}[dtype]
    c = Calls(dtype)
    c.cache = ms.kv_cache(**tensors(other, "cuda"))
    refused(c.all(), "the cache does not have")
    c = Calls(dtype)
    refused(c.all(ws=torch.zeros(c.ws.numel(), dtype=torch.uint8)), "ws must be on the GPU")
    for kw in ({}, dict(n=N + 3), dict(rows=R + 2)):
        c = Calls(dtype, **kw)
        for call in c.all():
            call()
        torch.cuda.synchronize()
        assert ms.read_device_error(c.ws) == ms.OK


def test_the_comparison_itself():
    """As above without a GPU: the struct's record against dims and R."""
    kd = ms.KvDims(Hq=2 * HKV, Hkv=HKV, D=D, page=PAGE, n_pages=N, max_pages=MAX, dtype=ms.FP8)
    c = ms.KvCache(0, 0, 0, 0, 0)

    class Ws:
        is_cuda = True
    ms._fits(c, kd, R, Ws, "call")  # raw pointers
    good = (ms.FP8, HKV, PAGE, D, MAX, N, R)
    for i, bad in enumerate((ms.BF16, HKV + 1, 2 * PAGE, D + 64, MAX + 1, N - 1, R - 1)):
        h = good[:i] + (bad,) + good[i + 1:]
        c._holds, c._n_pages, c._rows = h[:5], h[5], h[6]
        refused([lambda: ms._fits(c, kd, R, Ws, "call")], "call: the cache does not have")
    for more in (0, 1):
        c._holds, c._n_pages, c._rows = good[:5], N + more, R + more
        ms._fits(c, kd, R, Ws, "call")


@pytest.mark.parametrize("window,n_q,code", [(2 ** 31 - 257, 300, ms.EUNSUPPORTED), (2 ** 31 - 300, 300, ms.EUNSUPPORTED),
                                             (2 ** 31 - 301, 300, None), (2 ** 31 - 256, 300, None),
                                             (2 ** 31 - 1, 300, None), (2 ** 31 - 257, 256, None)])
def test_windows_that_pass_32_bits(window, n_q, code):
    """At the C entry, with a workspace too small: what is not refused for the window is refused for that."""
    kd = ms.KvDims(Hq=1, Hkv=1, D=D, page=16, n_pages=N, max_pages=(1 << 27) - 16)
    c = ms.KvCache(1 << 20, 1 << 20, None, None, 1 << 20)
    got = ms.lib().block_attention(kd._c, 1, n_q, 1 << 20, D, 1 << 20, c, 1.0, 0, window, 1 << 20, None, 1 << 20, 512, None)
    assert got == (ms.EWORKSPACE if code is None else code)


ATTENTION = [("q", torch.float16, "q must be"), ("q", torch.int16, "q must be"), ("q", torch.float64, "q must be"),
             ("out", torch.float16, "out must be"), ("out", torch.int16, "out must be"),
             ("n", torch.float32, "kv_len must be"), ("n", torch.int64, "kv_len must be"),
             ("lse", torch.int32, "lse must be"), ("lse", torch.bfloat16, "lse must be")]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [ms.BF16, ms.F32, ms.FP8])
def test_attention_takes_no_other_type(dtype):
    """One argument at a time, the others as they should be."""
    c = Calls(dtype)
    c.all()[2]()
    for name, other, match in ATTENTION:
        c = Calls(dtype)
        setattr(c, name, getattr(c, name).to(other))
        refused([c.all()[2]], f"block_attention: {match}")
    for name in ("q", "out", "n", "lse"):
        c = Calls(dtype)
        setattr(c, name, getattr(c, name).cpu())
        refused([c.all()[2]], "must be on the GPU")
    torch.cuda.synchronize()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [ms.BF16, ms.F32, ms.FP8])
def test_copies_take_no_other_type(dtype):
    for name, other in (("k", torch.float16), ("v", torch.float16), ("k", torch.int32), ("pos", torch.int64),
                        ("pos", torch.float32)):
        c = Calls(dtype)
        setattr(c, name, getattr(c, name).to(other))
        refused(c.all()[:2], f"{name} must be")
        c = Calls(dtype)
        setattr(c, name, getattr(c, name).cpu())
        refused(c.all()[:2], "must be on the GPU")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [ms.BF16, ms.F32])
def test_the_norm_takes_no_other_type(dtype):
    d = ms.ModelDims(H=256, E=8, k=2, I=64, Is=64, V=128, dtype=dtype)
    act = torch.float32 if dtype == ms.F32 else torch.bfloat16

    def call(**kw):
        z = lambda *s, t=torch.float32: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
        a = dict(y=z(2, 256), h_in=z(2, 256), h_out=z(2, 256), x=z(2, 256, t=act), w_pre=z(256, t=act),
                 w_post=z(256, t=act), gate=z(256))
        for name, f in kw.items():
            a[name] = f(a[name])
        ms.block_residual_norm(d, **a)

    call()
    torch.cuda.synchronize()
    half = lambda t: t.half()  # noqa: E731
    wrong = torch.bfloat16 if dtype == ms.F32 else torch.float32
    for name in ("y", "h_in", "h_out", "x", "w_pre", "w_post", "gate"):
        refused([lambda: call(**{name: half})], f"{name}.* must be")
        refused([lambda: call(**{name: lambda t: t.cpu()})], "on the GPU")
    for name in ("x", "w_pre", "w_post"):
        refused([lambda: call(**{name: lambda t: t.to(wrong)})], f"{name}.* must be")
    for name in ("h_in", "h_out", "gate"):
        refused([lambda: call(**{name: lambda t: t.bfloat16()})], f"{name}.* must be")
