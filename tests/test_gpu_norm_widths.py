"""block_residual_norm at every width of its row (128, 256 and 512 threads) that the dims admit, against the oracle.

Bounds.  A thread adds at most 16 squares in turn (a rounding each for the square and the sum), a warp its 32
sums in 5 steps, a row its at most 16 warps in turn: 1 + 16 + 5 + 16 = 38 u, u = 2^-24.  Mean and eps 2 u, all
halved by the root: 20 u; root and reciprocal 2 u: r = 22 u of 1 / rms.  h' adds 3 products (w, 1 / rms, gate),
res_scale and the sum: 27 u of |h| + |added| =: b.  x: r, the error of h' in rms (the root mean square of b, over
rms), two products, b itself, and the rounding to x's type."""
import numpy as np
import pytest
import torch

import moe_expert_step_gb300 as ms
from oracle import kv_attention as KV
from tests.test_gpu_residual_norm import NP, U, dims, make

pytestmark = pytest.mark.gpu


WIDTHS = [128, 896, 1024, 1152, 2048, 2176, 4096, 4224, 6400]  # (fp32: any multiple of 8)
CASES = [(H, t) for H in WIDTHS for t in (ms.BF16, ms.F32)] + [(H, ms.F32) for H in (8, 24, 136, 1000, 2056, 4104, 6392)]


@pytest.mark.parametrize("H,dtype", CASES)
@pytest.mark.parametrize("ydt", [torch.float32, torch.bfloat16])
def test_widths(H, ydt, dtype):
    T, P, s, eps = 5, 2, np.float32(0.7), np.float32(1e-6)
    y, h0, gate, w_post, w_pre, act = make(T, H, P, ydt, dtype, seed=H)
    h, x = torch.empty_like(h0), torch.empty((T, H), dtype=act, device="cuda")
    ms.block_residual_norm(dims(H, P, dtype), y, h0, h, x, w_pre=w_pre, w_post=w_post, gate=gate, res_scale=0.7)
    oh, ox = KV.block_residual_norm(NP(y), NP(h0), NP(w_post), NP(gate), NP(w_pre), s, eps, P)
    b = 27 * U * (np.abs(NP(h0)) + np.abs(oh - NP(h0)))
    assert (np.abs(NP(h) - oh) <= b).all()
    rms = np.sqrt((oh * oh).mean(1, keepdims=True) + eps)
    half = 2.0 ** -8 if act == torch.bfloat16 else U
    rel = 24 * U + np.sqrt((b * b).mean(1, keepdims=True)) / rms + half
    assert (np.abs(NP(x) - ox) <= (np.abs(NP(w_pre)) * b / rms + rel * np.abs(ox)) * (1 + 2.0 ** -7)).all()


@pytest.mark.parametrize("H", [6408, 6528, 8064, 8192, 8320])
def test_wider_is_refused(H):
    y, h0, *_ = make(1, H, 1, torch.float32, ms.F32)
    with pytest.raises(ms.MoeStepError) as e:
        ms.block_residual_norm(dims(H, 1, ms.F32), y, h0, h0, None)
    assert e.value.code == ms.EUNSUPPORTED
