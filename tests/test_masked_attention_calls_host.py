"""Masked attention, key ranges and the norm with rotation without a GPU: what their sources may contain and what their
entry points refuse."""
import ctypes
import os
import random
import re
import shutil
import subprocess

import pytest
import torch

import tensor_transformer_mlp_gb300 as tp
from tensor_transformer_mlp_gb300 import _binding, _build

OK, INVALID, SHAPE, DTYPE, ALIGN, CUDA, TIMEOUT, WORKSPACE = range(8)
F32, BF16 = 0, 1
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


# ------------------------------------------------------------------------- tensors that overlap

OVERLAP_C = r"""
#include "overlap.h"
extern "C" int meet(const long long* a, const long long* b) {
  auto r = [](const long long* x) { return tpmlp::Region{(uintptr_t)x[0], x[1], x[2], x[3], x[4], x[5]}; };
  return tpmlp::overlap(r(a), r(b));
}
"""


@pytest.fixture(scope="module")
def meet(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("overlap")
    (d / "meet.cpp").write_text(OVERLAP_C)
    subprocess.run([cxx, "-std=c++17", "-shared", "-fPIC", "-I", _build.CSRC, "-o", str(d / "meet.so"), str(d / "meet.cpp")],
                   check=True)
    lib = ctypes.CDLL(str(d / "meet.so"))

    def call(a, b):
        six = ctypes.c_longlong * 6
        return bool(lib.meet(six(*a), six(*b)))
    return call


def _bytes_of(r):
    at, rows, row, heads, head, width = r
    return {at + i * row + h * head + c for i in range(rows) for h in range(heads) for c in range(width)}


def test_overlap_against_sets_of_bytes(meet):
    r = random.Random(0)
    seen = {True: 0, False: 0}
    for n in range(6000):
        def draw():
            heads, width = r.randint(1, 4), r.choice([0, 1, 3, 4, 8])
            head = r.randint(1, 12)
            return [r.randint(0, 60), r.randint(1, 5), r.randint(1, 40), heads, head, width]
        a, b = draw(), draw()
        if n % 2:                                    # one matrix's strides, as packed tensors have
            b[2], b[4] = a[2], a[4]
        elif n % 3 == 0:
            b[2] = a[2]
        want = bool(_bytes_of(a) & _bytes_of(b))
        assert meet(a, b) == want and meet(b, a) == want, (a, b)
        seen[want] += 1
    assert min(seen.values()) > 500


def test_overlap_of_large_tensors(meet):
    at, t, h, hd = 1 << 40, 8192, 64, 256                             # 64 heads of 128 bf16 columns
    packed = [[at + n * hd, t, 3 * h * hd, h, 3 * hd, hd] for n in range(3)]
    for i in range(3):
        for j in range(3):
            assert meet(packed[i], packed[j]) == (i == j)
    assert meet(packed[0], [at + 16, t, 3 * h * hd, h, 3 * hd, hd])   # a few columns off
    assert meet(packed[0], [at + hd - 16, t, 3 * h * hd, h, 3 * hd, hd])
    end = at + t * 3 * h * hd
    assert not meet(packed[2], [end, t, h * hd, h, hd, hd]) and meet(packed[2], [end - 16, t, h * hd, h, hd, hd])
    assert not meet(packed[0], [end - 2 * hd, 1, 1, 1, 1, 2 * hd])    # between the last q and the end: k and v
    assert meet(packed[0], [end - 3 * hd + 8, 1, 1, 1, 1, 4])
    major = [at, t, hd, h, t * hd, hd]                                # all tokens of a head, then the next head
    assert meet(major, [at + 5 * t * hd + 8, t, hd, h, t * hd, hd])
    assert meet(major, [at + 8 * hd, 16, h * hd, 2, hd, hd])
    assert not meet([at, 1 << 31, 1 << 32, 65535, 1 << 39, hd], [at + hd, 1 << 31, 1 << 32, 65535, 1 << 39, hd])


AT = [n << 40 for n in range(1, 16)]       # never dereferenced: every call fails validation first
GOOD = (256, 64, 128, 64, 256, 64, 128, 64)


@pytest.fixture(scope="module")
def lib():
    return _binding.load_library(build_if_missing=True)


def _message(lib, status, code, text):
    assert status == code and text in lib.tpmlp_last_error().decode(), (status, lib.tpmlp_last_error())


def _ranges(lib, ids=AT[0], prefix=AT[1], causal=1, window=0, out=AT[2], b=2, s=16):
    return lib.tpmlp_attention_key_ranges(ids, prefix, causal, window, out, b, s, None)


def _forward(lib, q=AT[0], k=AT[1], v=AT[2], rng=AT[3], slopes=AT[4], scale=0.1, cap=0.0, o=AT[5], lse=AT[6], b=2, s=16,
             heads=4, kv=2, hd=64, st=GOOD[:4] + (128, 64, 256, 64), dt=BF16):
    return lib.tpmlp_masked_attention_forward(q, k, v, rng, slopes, scale, cap, o, lse, b, s, heads, kv, hd, *st, dt, None)


BACKWARD = GOOD[:4] + (128, 64) + GOOD[:2] + GOOD[:4] + (128, 64)


def _backward(lib, q=AT[0], k=AT[1], v=AT[2], rng=AT[3], slopes=AT[4], scale=0.1, cap=0.0, o=AT[5], lse=AT[6], do=AT[7],
              dq=AT[8], dk=AT[9], dv=AT[10], b=2, s=16, heads=4, kv=2, hd=64, st=BACKWARD, dt=BF16, ws=AT[11], wsb=1 << 20):
    return lib.tpmlp_masked_attention_backward(q, k, v, rng, slopes, scale, cap, o, lse, do, dq, dk, dv, b, s, heads, kv, hd,
                                               *st, dt, ws, wsb, None)


def _rope(lib, q=AT[0], k=AT[1], gq=AT[2], gk=AT[3], eps=1e-5, cos=AT[4], sin=AT[5], pos=AT[6], table=8, rot=64, style=0,
          qo=AT[7], ko=AT[8], b=1, s=8, heads=4, kv=2, hd=64, st=GOOD, dt=BF16):
    return lib.tpmlp_qk_norm_rope(q, k, gq, gk, eps, cos, sin, pos, table, rot, style, qo, ko, b, s, heads, kv, hd, *st, dt,
                                  None)


def _rope_backward(lib, q=AT[0], k=AT[1], gq=AT[2], gk=AT[3], eps=1e-5, cos=AT[4], sin=AT[5], pos=AT[6], table=8, rot=64,
                   style=0, dqo=AT[7], dko=AT[8], dq=AT[9], dk=AT[10], dgq=AT[11], dgk=AT[12], b=1, s=8, heads=4, kv=2, hd=64,
                   st=GOOD + GOOD[4:], dt=BF16, ws=AT[13], wsb=1 << 20):
    return lib.tpmlp_qk_norm_rope_backward(q, k, gq, gk, eps, cos, sin, pos, table, rot, style, dqo, dko, dq, dk, dgq, dgk, b,
                                           s, heads, kv, hd, *st, dt, ws, wsb, None)


@pytest.mark.parametrize("call,outputs,others", [
    (_ranges, "out", "ids prefix"),
    (_forward, "o lse", "q k v rng slopes"),
    (_backward, "dq dk dv ws", "q k v rng slopes o lse do"),
    (_rope, "qo ko", "q k gq gk cos sin pos"),
    (_rope_backward, "dq dk dgq dgk ws", "q k gq gk cos sin pos dqo dko")])
def test_outputs_that_lie_across_other_tensors_are_refused(lib, call, outputs, others):
    place = dict(zip(call.__code__.co_varnames[1:call.__code__.co_argcount], call.__defaults__))
    for out in outputs.split():
        for other in (outputs + " " + others).split():
            if other != out:     # 256 bytes into it (what is smaller than that: from its start)
                off = 0 if other in ("gq", "gk", "slopes", "prefix", "dgq", "dgk", "ids", "pos", "rng", "lse") else 256
                if out == "ws" and other in ("gq", "gk", "slopes"):
                    off = 0
                _message(lib, call(lib, **{out: place[other] + off}), INVALID, "overlaps")


def test_a_few_columns_off_in_a_packed_matrix_are_refused(lib):
    packed, heads = (768, 192), dict(heads=4, kv=4)
    qkv = dict(q=AT[0], k=AT[0] + 128, v=AT[0] + 256)
    _message(lib, _forward(lib, **qkv, **heads, st=packed * 4, o=AT[0] + 256 - 16), INVALID, "overlaps")
    _message(lib, _backward(lib, **qkv, **heads, dq=AT[8], dk=AT[8] + 128, dv=AT[8] + 256 - 16,
                            st=packed * 3 + (256, 64) + packed * 3), INVALID, "overlaps")
    _message(lib, _rope(lib, q=AT[0], k=AT[0] + 128, qo=AT[0], ko=AT[0] + 256 - 16, **heads, st=packed * 4), INVALID,
             "overlaps")


@pytest.mark.skipif(torch.cuda.is_available(), reason="without a device an accepted call ends where it looks for one")
def test_one_packed_matrix_may_hold_all_inputs_or_all_gradients(lib):
    packed, heads = (768, 192), dict(heads=4, kv=4)
    qkv = dict(q=AT[0], k=AT[0] + 128, v=AT[0] + 256)
    for call in (lambda: _forward(lib, **qkv, **heads, st=packed * 3 + (256, 64)),
                 lambda: _forward(lib, q=AT[0], k=AT[1], v=AT[1], **heads, st=(256, 64) * 4),      # inputs may be shared
                 lambda: _backward(lib, **qkv, **heads, dq=AT[8], dk=AT[8] + 128, dv=AT[8] + 256,
                                   st=packed * 3 + (256, 64) + packed * 3),
                 lambda: _rope(lib, q=AT[0], k=AT[0] + 128, qo=AT[0], ko=AT[0] + 128, **heads, st=packed * 4),
                 lambda: _rope(lib, qo=AT[8], ko=AT[8] + 128, **heads, st=(256, 64, 256, 64) + packed * 2),
                 lambda: _rope_backward(lib, q=AT[0], k=AT[0] + 128, dq=AT[0], dk=AT[0] + 128, **heads,
                                        st=packed * 2 + (256, 64) * 2 + packed * 2),
                 lambda: _rope_backward(lib, dq=AT[7], dk=AT[8]),
                 lambda: _ranges(lib), lambda: _rope(lib), lambda: _rope_backward(lib), lambda: _forward(lib),
                 lambda: _backward(lib)):
        assert call() == CUDA


# ------------------------------------------------------------------------- the Python functions

def test_rope_tables_of_odd_widths_are_refused():
    # 7 columns would get a table of 4 pairs, and the norm with rotation would then turn 8 by other angles
    for rot in (7, 1, 0, -2):
        with pytest.raises(ValueError, match="rot_dim must be even"):
            tp.rope_tables(16, rot)
    cos, sin = tp.rope_tables(16, 6)
    assert cos.shape == sin.shape == (16, 3)


def test_key_ranges_on_another_device_than_their_tensors_are_refused():
    ids, prefix = torch.zeros(1, 8, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for kw in (dict(doc_ids=ids), dict(prefix_len=prefix), dict(doc_ids=ids, prefix_len=prefix)):
        for device in ("cuda", "cuda:1", torch.device("cuda", 0)):
            with pytest.raises(ValueError, match="on cpu, not on cuda"):
                tp.attention_key_ranges(1, 8, device=device, **kw)
        with pytest.raises(ValueError, match="must be CUDA tensors"):
            tp.attention_key_ranges(1, 8, device="cpu", **kw)
