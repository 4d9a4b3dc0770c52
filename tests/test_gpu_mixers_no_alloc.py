"""The planning, rotary and delta-rule calls allocate no memory, neither through torch nor of the device."""
import pytest
import torch

import moe_expert_step_gb300 as ms

pytestmark = pytest.mark.gpu


def test_calls_allocate_nothing():
    R, n = 80, 140
    z = lambda *s, t=torch.bfloat16: torch.randn(s, device="cuda").to(t)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    kd = ms.KvDims(Hq=4, Hkv=2, D=64, page=16, n_pages=R, max_pages=10)
    ring, head = torch.arange(R, dtype=torch.int32, device="cuda"), torch.tensor([0, R], dtype=torch.int32, device="cuda")
    plan = (i32(R), i32(R), ring, head, head, i32(R, 10), i32(R), i32(R, n), ms.kv_workspace(kd, R, 1))
    q, k, freq, pos = z(R * n, 4, 64), z(R * n, 2, 64), ms.rotary_frequencies(64, 1e4), i32(R, n)
    deltas = []
    for m, dtype in ((1, ms.BF16), (20, ms.F32), (32, ms.BF16), (n, ms.BF16)):  # by tokens, a short chunk, whole heads
        for few in (2, R):
            dd, act = ms.DeltaDims(Hk=1, Hv=2, Dk=64, Dv=128, n_slots=few, dtype=dtype), torch.float32 if dtype else torch.bfloat16
            T, f = few * m, torch.float32
            S = torch.zeros((few, 2, 128, 64), device="cuda")
            deltas.append(((dd, few, z(T, 1, 64, t=act), z(T, 1, 64, t=act), z(T, 2, 128, t=act), -z(T, 2, t=f).abs(),
                            z(T, 2, t=f).sigmoid(), S, z(T, 2, 128, t=act), ms.delta_workspace(dd, few, m)), S))

    def calls():
        ms.kv_cache_plan(kd, R, *plan)
        ms.block_rotary(kd, q, k, pos, freq, q, k)
        for a, S in deltas:
            ms.block_delta_rule(*a, state_out=S, qk_eps=1e-6)
        torch.cuda.synchronize()

    calls()  # (the first one loads the kernels)
    count = lambda: torch.cuda.memory_stats()["allocation.all.allocated"]  # noqa: E731
    before, free = count(), torch.cuda.mem_get_info()[0]
    for _ in range(3):
        calls()
    assert count() == before
    assert torch.cuda.mem_get_info()[0] >= free
