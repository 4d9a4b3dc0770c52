"""The example decoder: the cache, attention, residual norms and the MoE step run together."""
import numpy as np
import pytest
import torch

import moe_expert_step_gb300 as ms
from examples.block_decoder import small
from oracle import kv_attention as KV
from tests.helpers import BF16_TOL, max_rel

pytestmark = pytest.mark.gpu
NP = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("P,prefix", [(32, 100), (1, 37), (8, 0)])
def test_attention_sublayer_against_float64(fp8, P, prefix):
    """Each layer's attention half, from the layer's own input and cache, in float64: the residual
    stream to the bf16 tolerance of the whole step (projections round to bf16 on the way)."""
    m = small(2, prefix, 1, fp8, P)
    rec = []
    m.forward(rec)
    torch.cuda.synchronize()
    m.check()
    d, kd, n = m.d, m.kd, prefix + P
    pos = torch.arange(n, dtype=torch.int32, device="cuda").repeat(2, 1)
    for L, r in zip(m.layers, rec):
        k, v = (torch.empty((2 * n, kd.Hkv, kd.D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
        ms.kv_cache_read(kd, 2, pos, L.cache, k, v, m.kv_ws)
        k, v = NP(k).reshape(2, n, kd.Hkv, kd.D), NP(v).reshape(2, n, kd.Hkv, kd.D)
        qkv = (NP(r["x"]) @ NP(L.Wqkv).T).reshape(2 * P, -1, kd.D)
        step = 2.0 ** -3 if fp8 else 2.0 ** -7
        new = qkv[:, kd.Hq:kd.Hq + kd.Hkv].reshape(2, P, kd.Hkv, kd.D)
        assert np.abs(k[:, prefix:] - new).max() <= step * np.abs(new).max()   # the block itself is in the cache
        out, _, _, _ = KV.block_attention(qkv[:, :kd.Hq], list(k), list(v), [n, n], P, kd.D ** -0.5, False, 0)
        y = out.reshape(2 * P, -1) @ NP(L.Wo).T
        h, x = KV.block_residual_norm(y, NP(r["h"]), NP(L.attn_out), NP(m.gate), NP(L.moe_in), 1.0, 1e-6, P)
        assert max_rel(NP(r["h_mid"]), h) <= BF16_TOL
        assert max_rel(NP(r["x_mid"]), x) <= BF16_TOL


@pytest.mark.parametrize("fp8", [False, True])
def test_blocks_resolve_and_repeat(fp8):
    """Every block resolves within P rounds, the prefix grows, and a second run gives the same tokens."""
    runs = []
    for _ in range(2):
        m = small(2, 50, 2, fp8, seed=3)
        toks, rounds = [], []
        for _ in range(2):
            rounds.append(m.decode_block(logit_scale=8.0))
            toks.append(m.tokens.clone())
            assert not m.masked.any() and 1 <= rounds[-1] <= m.d.P
        m.check()
        assert m.kv_len.tolist() == [50 + 2 * m.d.P] * 2
        runs.append((rounds, torch.stack(toks)))
    assert runs[0][0] == runs[1][0] and torch.equal(runs[0][1], runs[1][1])
    assert int(runs[0][1].max()) < 4096 and int(runs[0][1].min()) >= 0
