"""Tensor memory and programmatic dependent launch (CPU, on the kernels' sources).

A kernel lets its successor start (pdl_trigger) while its own blocks run, and a successor may take tensor memory before it waits
for the kernel (pdl_wait).  A block that had triggered but not taken its tensor memory yet could then wait for memory that
the successor gives back only after that block has ended.  So a kernel that takes tensor memory has it in every thread's
sight (a barrier) before it triggers."""
import glob
import os
import re

import pytest

import moe_expert_step_gb300 as ms

CSRC = os.path.join(os.path.dirname(ms.__file__), "csrc")
KERNELS = []
for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
    text = re.sub(r"//[^\n]*", "", open(path).read())
    for part in re.split(r"(?=__global__ void)", text)[1:]:
        if "tmem_alloc(" in part:
            KERNELS.append((os.path.basename(path), part))


def test_the_kernels_are_found():
    assert {name for name, _ in KERNELS} == {"attention_tc.cu", "delta_heads.cu", "expert_gemm.cu"}


@pytest.mark.parametrize("name,body", KERNELS, ids=[k[0] for k in KERNELS])
def test_tensor_memory_is_taken_before_the_successor_may_start(name, body):
    alloc, trigger = body.index("tmem_alloc("), body.index("pdl_trigger()")
    assert alloc < body.index("__syncthreads()", alloc) < trigger
    assert body.count("pdl_trigger()") == 1
