"""The example decoder with pages planned on the GPU, rotary positions and the gated delta rule: the three operators
run together with the cache, attention and the MoE step."""
import numpy as np
import pytest
import torch

import moe_expert_step_gb300 as ms
from examples.block_decoder import hybrid
from oracle import kv_attention as KV
from oracle import token_mixer as TM
from tests.helpers import BF16_TOL, max_rel

pytestmark = pytest.mark.gpu
NP = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731


def delta_reference(m, M, x, state):
    """(mixer's output, new states) of layer inputs x [T, H] in float64."""
    dd, P = m.dd, m.d.P
    at = np.cumsum((0,) + m.widths)
    q, k, v, a, b = ((NP(x) @ NP(M["Win"]).T)[:, at[i]:at[i + 1]] for i in range(5))
    g = -NP(M["rate"]) * np.log1p(np.exp(a))
    beta = 1 / (1 + np.exp(-b))
    outs, states = [], []
    for r in range(m.R):
        s = slice(r * P, (r + 1) * P)
        o, S, _ = TM.delta_rule(q[s].reshape(P, dd.Hk, dd.Dk), k[s].reshape(P, dd.Hk, dd.Dk), v[s].reshape(P, dd.Hv, dd.Dv),
                                g[s], beta[s], NP(state[r]), dd.Dk ** -0.5, 1e-6)
        outs.append(o.reshape(P, -1))
        states.append(S)
    return np.concatenate(outs) @ NP(M["Wout"]).T, np.stack(states)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("P", [32, 8, 64])
def test_mixers_against_float64(fp8, P):
    """After a resolved block, the second block's pass: each layer's token mixer from the layer's own input, its history
    and its cache, in float64; then the states that take the block in."""
    m = hybrid(3, 2, fp8, P)
    m.decode_block(logit_scale=8.0)
    m.begin()
    assert m.seen.tolist() == [2 * P] * 3 and m.pos[1].tolist() == list(range(P, 2 * P))
    used = m.table[m.table >= 0].tolist()
    assert len(set(used)) == len(used) == 3 * -(-2 * P // 16)
    m.masked.fill_(1)
    before = {i: M["state"].clone() for i, M in m.delta.items()}
    rec = []
    m.forward(rec, resolved=True)
    torch.cuda.synchronize()
    m.check()
    kd, n = m.kd, 2 * P
    pos = torch.arange(n, dtype=torch.int32, device="cuda").repeat(3, 1)
    radians = TM.rotary_frequencies(kd.D // 2, 1e4)
    for i, (L, r) in enumerate(zip(m.layers, rec)):
        if i in m.delta:
            y, S = delta_reference(m, m.delta[i], r["x"], before[i])
            # the projections' bf16 rounding (2^-8 of each input) through a contraction of at most P tokens
            assert max_rel(NP(m.delta[i]["state"]), S) <= BF16_TOL
        else:
            k, v = (torch.empty((3 * n, kd.Hkv, kd.D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
            ms.kv_cache_read(kd, 3, pos, L.cache, k, v, m.kv_ws)
            k, v = NP(k).reshape(3, n, kd.Hkv, kd.D), NP(v).reshape(3, n, kd.Hkv, kd.D)
            qkv = (NP(r["x"]) @ NP(L.Wqkv).T).reshape(3 * P, -1, kd.D)
            places = m.pos.reshape(-1).tolist()
            q, _ = TM.block_rotary(qkv[:, :kd.Hq], places, radians, False, 1.0)
            new, _ = TM.block_rotary(qkv[:, kd.Hq:kd.Hq + kd.Hkv], places, radians, False, 1.0)
            new = new.reshape(3, P, kd.Hkv, kd.D)
            step = 2.0 ** -3 if fp8 else 2.0 ** -6  # two bf16 roundings (projection, rotation), or E4M3's
            assert np.abs(k[:, P:] - new).max() <= step * np.abs(new).max()
            out, _, _, _ = KV.block_attention(q, list(k), list(v), [n] * 3, P, kd.D ** -0.5, False, 0)
            y = out.reshape(3 * P, -1) @ NP(L.Wo).T
        h, x = KV.block_residual_norm(y, NP(r["h"]), NP(L.attn_out), NP(m.gate), NP(L.moe_in), 1.0, 1e-6, P)
        assert max_rel(NP(r["h_mid"]), h) <= BF16_TOL
        assert max_rel(NP(r["x_mid"]), x) <= BF16_TOL


def test_blocks_resolve_end_and_repeat():
    """Blocks resolve, all pages come back at the end, and a second run from nothing gives the same tokens."""
    m = hybrid(2, 2, False, seed=5)
    runs = []
    for _ in range(2):
        toks = []
        for _ in range(2):
            before = {i: M["state"].clone() for i, M in m.delta.items()}
            assert 1 <= m.decode_block(logit_scale=8.0) <= m.d.P
            assert all(not torch.equal(before[i], M["state"]) for i, M in m.delta.items())
            toks.append(m.tokens.clone())
            assert not m.masked.any()
        runs.append(torch.stack(toks))
        m.end()
        m.check()
        for M in m.delta.values():
            M["state"].zero_()
    assert torch.equal(*runs)


def test_a_history_is_left_until_the_block_is_resolved():
    m = hybrid(2, 2, False, seed=7)
    m.decode_block(logit_scale=8.0)
    m.begin()
    m.masked.fill_(1)
    before = {i: M["state"].clone() for i, M in m.delta.items()}
    m.forward()
    first = m.h.clone()
    m.forward()
    assert torch.equal(first, m.h) and all(torch.equal(before[i], M["state"]) for i, M in m.delta.items())
    m.forward(resolved=True)
    assert torch.equal(first, m.h) and all(not torch.equal(before[i], M["state"]) for i, M in m.delta.items())
    m.check()


def test_pages_come_back():
    m = hybrid(2, 3, True, seed=6)
    for _ in range(3):
        m.decode_block(logit_scale=8.0)
    assert m.head.tolist()[1] == 1
    m.end()
    first, count = m.head.tolist()
    assert count == m.kd.n_pages
    assert sorted(m.ring.tolist()) == list(range(m.kd.n_pages))
    for _ in range(3):  # and serve again
        m.decode_block(logit_scale=8.0)
    m.check()
    assert m.kv_len.tolist() == [3 * m.d.P] * 2 and m.head.tolist()[1] == 1
