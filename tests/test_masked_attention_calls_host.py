"""Masked attention, key ranges and the norm with rotation without a GPU: what their sources may contain and what their
entry points refuse."""
import os
import re

import pytest

from tensor_transformer_mlp_gb300 import _build

KERNELS = ["masked_attention_fwd.cu", "masked_attention_bwd.cu", "attention_tiles.cuh", "device_common.cuh"]


@pytest.mark.parametrize("name", KERNELS)
def test_no_wait_without_a_limit(name):
    # A role of a kernel that gives up returns, so the others may wait for it only where the wait has a limit, or at the
    # barrier that every role reaches on its way out.
    with open(os.path.join(_build.CSRC, name)) as f:
        source = re.sub(r"//[^\n]*", "", f.read())
    assert not re.search(r"\bbar(rier)?(\.cta)?\.(sync|red)", source)
    for kernel in source.split("__global__")[1:]:
        assert "__syncthreads" not in kernel.split("regs_dec<")[-1].split("tc_fence_before();\n  __syncthreads();")[0]
