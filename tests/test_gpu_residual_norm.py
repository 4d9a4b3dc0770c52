"""block_residual_norm against the oracle.

Bounds, elementwise.  A sum of squares of H fp32 terms held by 256 threads and joined in trees errs
relatively by less than (H / 256 + 16) u with u = 2^-24, half of that after the square root; the
norm's product and division add 4 u, the gate, scale and addition 3 u of their terms.  With H <= 6400
everything stays below 32 u of |h| + |res_scale * gate * w * y / rms|.  x inherits that of h, relative to
rms(h) = 1 after the norm, and is rounded once to its own type."""
import numpy as np
import pytest
import torch

import moe_expert_step_gb300 as ms
from oracle import kv_attention as KV

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
NP = lambda t: None if t is None else t.float().cpu().numpy().astype(np.float64)  # noqa: E731


def dims(H, P, dtype):
    return ms.ModelDims(H=H, E=256, k=8, I=512, Is=512, V=1000, P=P, dtype=dtype)


def make(T, H, P, ydt, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    act = torch.float32 if dtype == ms.F32 else torch.bfloat16
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return (r(T, H).to(ydt), 2 * r(T, H), r(-(-T // P), H), (1 + 0.1 * r(H)).to(act), (1 + 0.1 * r(H)).to(act), act)


def check(h, x, y, h0, w_post, gate, w_pre, s, eps, P, act):
    oh, ox = KV.block_residual_norm(NP(y), NP(h0), NP(w_post), NP(gate), NP(w_pre), s, eps, P)
    added = np.abs(oh - NP(h0))
    bound = 32 * U * (np.abs(NP(h0)) + added) + 1e-30
    assert (np.abs(NP(h) - oh) <= bound).all()
    if x is None:
        return
    rms = np.sqrt((oh * oh).mean(1, keepdims=True) + eps)
    w = 1.0 if w_pre is None else np.abs(NP(w_pre))
    half = 2.0 ** -8 if act == torch.bfloat16 else U
    bx = w * (bound / rms) + (32 * U + half) * np.abs(ox) + 1e-30
    assert (np.abs(NP(x) - ox) <= bx).all()


@pytest.mark.parametrize("T,H,P", [(1, 128, 1), (5, 256, 2), (32, 2048, 32), (33, 2048, 8), (7, 1280, 3),
                                   (3, 5120, 1), (2, 6400, 32), (300, 640, 64)])
@pytest.mark.parametrize("ydt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dtype", [ms.BF16, ms.F32])
def test_against_the_oracle(T, H, P, ydt, dtype):
    y, h0, gate, w_post, w_pre, act = make(T, H, P, ydt, dtype)
    h, x = torch.empty_like(h0), torch.empty((T, H), dtype=act, device="cuda")
    ms.block_residual_norm(dims(H, P, dtype), y, h0, h, x, w_pre=w_pre, w_post=w_post, gate=gate, res_scale=0.7)
    check(h, x, y, h0, w_post, gate, w_pre, np.float32(0.7), np.float32(1e-6), P, act)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("gated", ["no", "one", "one row", "strided"])
def test_optional_parts(post, pre, gated):
    T, H, P = 9, 512, 4
    y, h0, gate, w_post, w_pre, act = make(T, H, P, torch.float32, ms.BF16, 1)
    wide = torch.zeros((3, 2 * H), device="cuda")
    wide[:, :H] = gate
    g = {"no": None, "one": gate[0], "one row": gate[:1].expand(3, H), "strided": wide[:, :H]}[gated]
    h, x = torch.empty_like(h0), torch.empty((T, H), dtype=act, device="cuda")
    a = dict(w_pre=w_pre if pre else None, w_post=w_post if post else None, gate=g)
    ms.block_residual_norm(dims(H, P, ms.BF16), y, h0, h, x, **a)
    check(h, x, y, h0, a["w_post"], None if g is None else g if g.dim() == 1 else g.contiguous(), a["w_pre"], 1.0,
          np.float32(1e-6), P, act)


def test_in_place_and_without_x():
    T, H, P = 6, 1024, 2
    y, h0, gate, w_post, w_pre, act = make(T, H, P, torch.bfloat16, ms.BF16, 2)
    h, h2, x = torch.empty_like(h0), h0.clone(), torch.empty((T, H), dtype=act, device="cuda")
    ms.block_residual_norm(dims(H, P, ms.BF16), y, h0, h, x, w_pre=w_pre, w_post=w_post, gate=gate)
    ms.block_residual_norm(dims(H, P, ms.BF16), y, h2, h2, None, w_post=w_post, gate=gate)
    assert torch.equal(h, h2)


def test_zero_and_infinite_rows():
    """A row of zeros stays finite (eps); a non-finite one touches no other row."""
    T, H = 4, 256
    y, h0, _, w_post, w_pre, act = make(T, H, 1, torch.float32, ms.BF16, 3)
    y[1], h0[1] = 0.0, 0.0
    y[2, 3] = float("inf")
    h, x = torch.empty_like(h0), torch.empty((T, H), dtype=act, device="cuda")
    ms.block_residual_norm(dims(H, 1, ms.BF16), y, h0, h, x, w_pre=w_pre, w_post=w_post)
    assert not h[1].any() and not x[1].any()
    rest = [0, 1, 3]
    assert torch.isfinite(h[rest]).all() and torch.isfinite(x[rest].float()).all()
    check(h[rest], x[rest], y[rest], h0[rest], w_post, None, w_pre, 1.0, np.float32(1e-6), 1, act)


def test_many_rows_are_rows_of_few():
    """Each token's result does not depend on how many there are."""
    y, h0, gate, w_post, w_pre, act = make(5000, 256, 10, torch.bfloat16, ms.BF16, 4)
    d = dims(256, 10, ms.BF16)
    h, x = torch.empty_like(h0), torch.empty((5000, 256), dtype=act, device="cuda")
    ms.block_residual_norm(d, y, h0, h, x, w_pre=w_pre, w_post=w_post, gate=gate)
    hs, xs = torch.empty_like(h0[:10]), torch.empty_like(x[:10])
    for t in (0, 2490, 4990):
        ms.block_residual_norm(d, y[t:t + 10], h0[t:t + 10], hs, xs, w_pre=w_pre, w_post=w_post,
                               gate=gate[t // 10:t // 10 + 1])
        assert torch.equal(hs, h[t:t + 10]) and torch.equal(xs, x[t:t + 10])
