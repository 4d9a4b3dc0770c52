"""kv_cache_plan on workspaces that other calls use between its own."""
import numpy as np
import pytest
import torch

import moe_expert_step_gb300 as ms
from oracle import token_mixer as om
from tests.test_gpu_kv_plan import call, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,n", [(300, 50), (3, 4096), (1, 32)])
def test_in_place_on_the_workspace_of_the_moe_step(R, n):
    """The header is updated in place after a router call has left its counters in the same workspace."""
    d = ms.ModelDims(H=512, E=32, k=4, I=128, Is=128, V=4096)
    kd, *state = make(R, n, 16, 77 + R)
    want = om.kv_cache_plan(state[0], state[1], n, *state[2:], 16)
    ws = ms.workspace(d, 8)
    x, Wr = torch.randn((8 * d.P, d.H), device="cuda").bfloat16(), torch.randn((d.E, d.H), device="cuda").bfloat16()
    idx = torch.empty((8 * d.P, d.k), dtype=torch.int32, device="cuda")
    mass, gate = torch.empty(idx.shape, device="cuda"), torch.empty(idx.shape, device="cuda")
    n_sel, sel = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((8,), (8, d.E)))
    survive, top_p = torch.empty(idx.shape, dtype=torch.uint8, device="cuda"), torch.full((8,), 0.9, device="cuda")
    for _ in range(3):
        ms.moe_block_route(d, x, Wr, idx, mass, gate, ws)
        ms.coreset_select(d, 8, top_p, idx, mass, n_sel, sel, survive, gate, ws)
        got, word = call(kd, *state, n, ws=ws, in_place=True)
        check(got, want)
        assert word == ms.OK


def test_in_place_among_the_attention_side_and_the_delta_rule():
    """One workspace large enough for all of them, each call in turn."""
    R, n, page = 40, 64, 16
    kd, *state = make(R, n, page, 5)
    want = om.kv_cache_plan(state[0], state[1], n, *state[2:], page)
    dd = ms.DeltaDims(Hk=1, Hv=2, Dk=64, Dv=64, n_slots=R)
    size = max(ms.kv_workspace_size(kd, R, n), ms.delta_workspace_size(dd, R, n))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    ms.workspace_init(ws)
    z = lambda *s, t=torch.bfloat16: torch.randn(s, device="cuda").to(t)  # noqa: E731
    q, k, v, f = z(R * n, 1, 64), z(R * n, 1, 64), z(R * n, 2, 64), torch.float32
    S, out = torch.zeros((R, 2, 64, 64), device="cuda"), z(R * n, 2, 64)
    pool = [z(kd.n_pages, 2, page, 64) for _ in "kv"]
    for _ in range(3):
        got, word = call(kd, *state, n, ws=ws, in_place=True)
        check(got, want)
        assert word == ms.OK
        ms.block_delta_rule(dd, R, q, k, v, -z(R * n, 2, t=f).abs(), z(R * n, 2, t=f).sigmoid(), S, out, ws, state_out=S,
                            qk_eps=1e-6)
        cache = ms.kv_cache(*pool, torch.as_tensor(np.ascontiguousarray(got[2])).to(torch.int32).cuda())
        att = z(R * n, 4, 64)
        ms.block_attention(kd, R, att.clone(), torch.as_tensor(got[3]).to(torch.int32).cuda().clamp(min=0), cache, att, ws, 0.125,
                           causal=True)
        assert ms.read_device_error(ws) == ms.OK


@pytest.mark.parametrize("R,n", [(300, 50), (3, 4096)])
def test_in_place_whatever_stands_behind_the_header_of_256_bytes(R, n):
    """What the MoE step keeps behind its workspace's header of 256 bytes (counters, which a call that timed out may leave
    anywhere) is nothing to the plan."""
    kd, *state = make(R, n, 16, 78 + R)
    want = om.kv_cache_plan(state[0], state[1], n, *state[2:], 16)
    ws = ms.kv_workspace(kd, R, 1)
    ws[256:] = 1
    behind = ws[256:].clone()
    for _ in range(3):
        got, word = call(kd, *state, n, ws=ws, in_place=True)
        check(got, want)
        assert word == ms.OK and torch.equal(ws[256:], behind)
