"""block_rotary and rotary_frequencies against float64.

Bound of a turned element, in units of 2^-24 (|x0| + |x1|) |mscale|: the half-turn that goes to sincospif is
rounded to 32 bits and then to a float, 2^-32 + 2^-25 half-turns at most, 1.6 units of angle; sincospif is off by at most
2 units; the multiplication by mscale, the products and the sum by one each: 6.6, and 8 are allowed.  In bf16 the
result is rounded once more, by 2^-8 of itself at most."""
import math

import numpy as np
import pytest
import torch

import moe_expert_step_gb300 as ms
from oracle import token_mixer as om

pytestmark = pytest.mark.gpu

SCALINGS = dict(plain=ms.ROTARY_PLAIN, linear=ms.ROTARY_LINEAR, rotations=ms.ROTARY_ROTATIONS,
                dimensions=ms.ROTARY_DIMENSIONS)


def dims(Hq, Hkv, D, dtype):
    return ms.KvDims(Hq=Hq, Hkv=Hkv, D=D, page=16, n_pages=1, max_pages=1, dtype=dtype)


def check(x, got, before, pos, freq, pairs, mscale):
    want, bound = om.block_rotary(x.double().cpu().numpy(), pos.reshape(-1).tolist(), freq, pairs, mscale)
    live = (pos.reshape(-1) >= 0).cpu()
    assert torch.equal(got.cpu()[~live], before.cpu()[~live])  # padding rows are left
    g, live = got.double().cpu().numpy(), live.numpy()
    tol = 8 * 2.0 ** -24 * bound + (2.0 ** -8 * np.abs(want) * (bound > 0) if x.dtype == torch.bfloat16 else 0.0)
    assert (np.abs(g - want)[live] <= (tol + 1e-300)[live]).all()


@pytest.mark.parametrize("scaling", list(SCALINGS))
@pytest.mark.parametrize("rot,base", [(128, 1e4), (64, 1e6), (32, 1e7), (2, 1e4), (24, 5e5), (128, 1.5)])
def test_frequencies(scaling, rot, base):
    kw = dict(factor=8.0, original=4096.0, low=1.0, high=32.0)
    got = ms.rotary_frequencies(rot, base, scaling=SCALINGS[scaling], **kw).cpu().numpy().view(np.uint64)
    want = om.rotary_frequencies(rot, base, scaling, **kw) / (2 * math.pi)
    # pow and the division of a double: a few units of 2^-53 of the value
    assert np.all(np.abs(got.astype(np.float64) * 2.0 ** -64 - want) <= 8 * 2.0 ** -53 * want + 2.0 ** -64)


@pytest.mark.parametrize("dtype", [ms.BF16, ms.F32])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("R,n,Hq,Hkv,D,rot", [(1, 1, 16, 2, 128, 128), (2, 5, 4, 4, 64, 64), (3, 7, 6, 2, 128, 32),
                                              (1, 33, 5, 1, 64, 16), (2, 3, 8, 1, 128, 24), (1, 4, 2, 2, 64, 2),
                                              (1, 9, 3, 3, 64, 62), (2, 2, 64, 8, 128, 126)])
def test_against_float64(dtype, pairs, R, n, Hq, Hkv, D, rot):
    g = torch.Generator(device="cuda").manual_seed(rot * 7 + n)
    act = torch.float32 if dtype == ms.F32 else torch.bfloat16
    row = torch.randn((R * n, Hq + 2 * Hkv, D), generator=g, device="cuda").to(act)
    pos = torch.randint(0, 2_000_000, (R, n), generator=g, device="cuda").to(torch.int32)
    pos[0, 0] = 0
    if n > 2:
        pos[-1, -1], pos[0, 1] = -1, 2 ** 31 - 1
    freq = ms.rotary_frequencies(rot, 1e6)
    radians = om.rotary_frequencies(rot, 1e6)
    kd, mscale = dims(Hq, Hkv, D, dtype), 1.25
    q, k = row[:, :Hq], row[:, Hq:Hq + Hkv]
    near = pos < 2_000_001
    posn = torch.where(near, pos, 12345)
    qo, ko = torch.full((R * n, Hq, D), 7.0, device="cuda").to(act), torch.full((R * n, Hkv, D), 7.0, device="cuda").to(act)
    before = qo.clone(), ko.clone()
    keep = row.clone()
    ms.block_rotary(kd, q, k, posn, freq, qo, ko, interleaved=pairs, mscale=mscale)
    check(q, qo, before[0], posn, radians, pairs, mscale)
    check(k, ko, before[1], posn, radians, pairs, mscale)
    assert torch.equal(row, keep)
    # in place, within the projection's rows: the same, and the values' part is not touched
    ms.block_rotary(kd, q, k, posn, freq, q, k, interleaved=pairs, mscale=mscale)
    live = posn.reshape(-1) >= 0
    assert torch.equal(q[live], qo[live]) and torch.equal(k[live], ko[live])
    assert torch.equal(row[:, Hq + Hkv:], keep[:, Hq + Hkv:]) and torch.equal(row[~live], keep[~live])
    # the last position that there is: |turn| is exact, so the length of a pair stays what it was
    ms.block_rotary(kd, keep[:, :Hq], None, torch.full_like(pos, 2 ** 31 - 1), freq, qo, None, interleaved=pairs)
    a, b = qo.double().square().sum(-1), keep[:, :Hq].double().square().sum(-1)
    assert ((a - b).abs() <= (2.0 ** -6 if dtype == ms.BF16 else 2.0 ** -19) * b).all()


@pytest.mark.parametrize("shift,ld_more", [(1, 0), (0, 3), (3, 5)])
def test_rows_without_alignment(shift, ld_more):
    """Rows that begin anywhere take the element-wise form, with the same values."""
    Hq, Hkv, D, T, rot = 4, 2, 64, 11, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((T, Hq, D), generator=g, device="cuda").bfloat16()
    pos = torch.arange(100, 100 + T, dtype=torch.int32, device="cuda").view(1, T)
    freq, kd = ms.rotary_frequencies(rot, 1e4), dims(Hq, Hkv, D, ms.BF16)
    want = torch.empty_like(x)
    ms.block_rotary(kd, x, None, pos, freq, want, None)
    ld = Hq * D + ld_more
    buf = torch.zeros(T * ld + shift, device="cuda").bfloat16()
    y = buf[shift:].view(T, ld)[:, :Hq * D].unflatten(1, (Hq, D)) if ld_more else buf[shift:].view(T, Hq, D)
    y.copy_(x)
    ms.block_rotary(kd, y, None, pos, freq, y, None)
    assert torch.equal(y, want)


def test_many_tokens_and_graph():
    """A size of many blocks equals the same rows in small calls; captured and replayed."""
    Hq, Hkv, D, R, n = 16, 2, 128, 3, 1500
    g = torch.Generator(device="cuda").manual_seed(9)
    q, k = torch.randn((R * n, Hq, D), generator=g, device="cuda").bfloat16(), torch.randn((R * n, Hkv, D), generator=g, device="cuda").bfloat16()
    pos = torch.arange(R * n, dtype=torch.int32, device="cuda").view(R, n) * 37
    freq, kd = ms.rotary_frequencies(D, 1e6), dims(Hq, Hkv, D, ms.BF16)
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    graph = torch.cuda.CUDAGraph()
    ms.block_rotary(kd, q, k, pos, freq, qo, ko)
    a, b = qo.clone(), ko.clone()
    qo.zero_()
    with torch.cuda.graph(graph):
        ms.block_rotary(kd, q, k, pos, freq, qo, ko)
    graph.replay()
    assert torch.equal(a, qo) and torch.equal(b, ko)
    for t in (0, 1499, 1500, 4499):
        o, p = torch.empty_like(q[:1]), torch.empty_like(k[:1])
        ms.block_rotary(kd, q[t:t + 1], k[t:t + 1], pos.view(-1)[t:t + 1].view(1, 1), freq, o, p)
        assert torch.equal(o[0], a[t]) and torch.equal(p[0], b[t])
