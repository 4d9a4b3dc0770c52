"""block_rotary at far positions, against angles reduced in whole numbers.

A table's entry f is a fraction of a turn times 2^64, so position p stands at exactly (p * f mod 2^64) / 2^64 turns; from there
float64 is exact enough.  Bound of a turned element, in units of 2^-24 (|x0| + |x1|) |mscale|: of the turn the upper 32 bits are
taken (2^-32 turns, 0.02 units of angle), held in a float (a half-turn is below 1, so off by 2^-25: 2^-26 turns, 1.6
units); sincospif is off by at most 2 units; mscale, the products and the sum by one each: 6.7, and 8 are allowed.  In bf16
the result is rounded once more, by 2^-8 of itself at most."""
import math

import numpy as np
import pytest
import torch

import moe_expert_step_gb300 as ms

pytestmark = pytest.mark.gpu

FAR = [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 30 + 1, 1_999_999_999, 16_777_217, 123_456_789, 2_000_001, 1, 0]


@pytest.mark.parametrize("dtype", [ms.BF16, ms.F32])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("D,rot,base,shift", [(128, 128, 1e4, 0), (64, 64, 1e7, 0), (128, 24, 1.5, 0), (64, 62, 1e6, 1)])
def test_far_positions(dtype, pairs, D, rot, base, shift):
    act, H, T = torch.float32 if dtype == ms.F32 else torch.bfloat16, 3, len(FAR)
    g = torch.Generator(device="cuda").manual_seed(rot)
    x = torch.empty(T * H * D + shift, device="cuda", dtype=act)[shift:].view(T, H, D)  # (shift: element by element)
    x.copy_(torch.randn((T, H, D), generator=g, device="cuda"))
    freq = ms.rotary_frequencies(rot, base)
    table = [int(f) for f in freq.cpu().numpy().view(np.uint64)]
    pos = torch.tensor([FAR], dtype=torch.int32, device="cuda")
    kd = ms.KvDims(Hq=H, Hkv=1, D=D, page=16, n_pages=1, max_pages=1, dtype=dtype)
    out, mscale = torch.empty_like(x), 0.75
    ms.block_rotary(kd, x, None, pos, freq, out, None, interleaved=pairs, mscale=mscale)
    got, x = out.double().cpu().numpy(), x.double().cpu().numpy()
    want, bound = x.copy(), np.zeros_like(x)
    half = rot // 2
    for t, p in enumerate(FAR):
        for i, f in enumerate(table):
            turn = (p * f % 2 ** 64) / 2 ** 64  # (whole numbers; one rounding to 53 bits)
            c, s = math.cos(2 * math.pi * turn), math.sin(2 * math.pi * turn)
            a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
            want[t, :, a] = mscale * (x[t, :, a] * c - x[t, :, b] * s)
            want[t, :, b] = mscale * (x[t, :, b] * c + x[t, :, a] * s)
            bound[t, :, a] = bound[t, :, b] = mscale * (np.abs(x[t, :, a]) + np.abs(x[t, :, b]))
    tol = 8 * 2.0 ** -24 * bound + (2.0 ** -8 * np.abs(want) * (bound > 0) if dtype == ms.BF16 else 0.0)
    assert (np.abs(got - want) <= tol).all()
