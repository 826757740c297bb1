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


@pytest.mark.parametrize("name", KERNELS[:2])
def test_the_wait_for_a_pieces_end_counts_from_its_last_progress(name):
    # A piece of work lasts as long as it has key tiles (2 s from 2^27 or so on), so its end may only be waited for that way.
    with open(os.path.join(_build.CSRC, name)) as f:
        source = f.read()
    assert len(re.findall(r"mbar_wait_moving\(ending, it & 1, k?v_full,", source)) == 1
    assert not re.search(r"mbar_(wait|poll)\(ending", source)


@pytest.mark.parametrize("name", KERNELS[:2])
def test_what_indexes_a_ring_does_not_go_negative(name):
    # A CTA's count of tiles has no bound (2^31 take some minutes), and its remainder is an address in shared memory.
    with open(os.path.join(_build.CSRC, name)) as f:
        source = re.sub(r"//[^\n]*", "", f.read())
    for kernel in source.split("__global__")[1:]:
        roles = kernel[kernel.index("regs_dec<"):]
        signed = re.findall(r"(?<!\()\bint ([^;{}()]*);", roles)            # declarations, but not a loop's own
        names = {part.split("=")[0].strip() for decl in signed for part in decl.split(",")}
        assert not names & {"n", "n0", "kn", "vn", "t", "st", "qs", "gs", "os"}
        assert not re.search(r"\[&\]\((int \w+, )?int [nkv]\b", roles)     # parameters that take them
        assert re.search(r"uint32_t (n|kn) = 0", roles)
