"""The planning, rotary and delta-rule calls launch on the current device, whose kernels cannot follow pointers of another one:
tensors elsewhere are refused before anything is launched.  (CPU: tensors that only say where they are.)"""
import pytest
import torch

import moe_expert_step_gb300 as ms

BF, I32, F32, I64, U8 = torch.bfloat16, torch.int32, torch.float32, torch.int64, torch.uint8


class Tensor:
    """What the binding asks of a tensor, on the GPU of index `device`."""
    is_cuda = True

    def __init__(self, device, dtype, *shape):
        self.device, self.dtype, self.shape = device, dtype, torch.Size(shape)

    def get_device(self):
        return self.device

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return 1

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


class Launched(Exception):
    pass


class Library:
    def moestep_error_string(self, code):
        return b"refused"

    def __getattr__(self, name):
        def call(*a):
            raise Launched
        return call


@pytest.fixture(params=[0, 1])
def current(request, monkeypatch):
    monkeypatch.setattr(ms, "_CURRENT", (lambda: request.param, lambda device: 0))
    monkeypatch.setattr(ms, "lib", Library)
    return request.param


KD = ms.KvDims(Hq=4, Hkv=2, D=64, page=16, n_pages=100, max_pages=8)
DD = ms.DeltaDims(Hk=2, Hv=4, Dk=128, Dv=64, n_slots=5)
PLAN = dict(kv_len=(I32, 3), n_new=(I32, 3), ring=(I32, 100), head=(I32, 2), head_out=(I32, 2), table=(I32, 3, 8),
            new_len=(I32, 3), pos=(I32, 3, 32), ws=(U8, 512), slots=(I32, 3, 32))
ROTARY = dict(q=(BF, 6, 4, 64), k=(BF, 6, 2, 64), pos=(I32, 2, 3), freq=(I64, 32), q_out=(BF, 6, 4, 64), k_out=(BF, 6, 2, 64))
DELTA = dict(q=(BF, 6, 2, 128), k=(BF, 6, 2, 128), v=(BF, 6, 4, 64), g=(F32, 6, 4), beta=(F32, 6, 4), state=(F32, 5, 4, 64, 128),
             out=(BF, 6, 4, 64), ws=(U8, 512), state_out=(F32, 5, 4, 64, 128), slot=(I32, 2), length=(I32, 2), fresh=(U8, 2))
CALLS = dict(kv_cache_plan=(PLAN, lambda t: ms.kv_cache_plan(KD, 3, **t)), block_rotary=(ROTARY, lambda t: ms.block_rotary(KD, **t)),
             block_delta_rule=(DELTA, lambda t: ms.block_delta_rule(DD, 2, **t)))


@pytest.mark.parametrize("name,elsewhere", [(n, x) for n, (ts, _) in CALLS.items() for x in ts])
def test_tensors_on_another_device_are_refused(current, name, elsewhere):
    kinds, call = CALLS[name]
    with pytest.raises(Launched):
        call({k: Tensor(current, *v) for k, v in kinds.items()})
    with pytest.raises(ms.MoeStepError, match="current device") as e:
        call({k: Tensor(1 - current if k == elsewhere else current, *v) for k, v in kinds.items()})
    assert e.value.code == ms.EINVAL and elsewhere in str(e.value)


def test_frequencies_on_another_device_are_refused(current, monkeypatch):
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: Tensor(device, dtype, n))
    with pytest.raises(Launched):
        ms.rotary_frequencies(64, 1e4, device=current)
    with pytest.raises(ms.MoeStepError, match="the current one"):
        ms.rotary_frequencies(64, 1e4, device=1 - current)
