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


# ------------------------------------------------------------------------- refusals, each by its own message

POINTERS = {_ranges: "ids? prefix? out", _forward: "q k v rng slopes? o lse", _backward: "q k v rng slopes? o lse do dq dk dv",
            _rope: "q k gq gk cos sin pos? qo ko", _rope_backward: "q k gq gk cos sin pos? dqo dko dq dk dgq dgk"}
FOURS = "ids prefix slopes lse gq gk cos sin pos dgq dgk".split()     # 4-byte aligned; ranges 8, tensors of heads 16


@pytest.mark.parametrize("call", list(POINTERS))
def test_pointers_are_looked_at(lib, call):
    place = dict(zip(call.__code__.co_varnames[1:call.__code__.co_argcount], call.__defaults__))
    for name in POINTERS[call].split():
        if not name.endswith("?"):
            _message(lib, call(lib, **{name: None}), INVALID, "null pointer")
        name = name.rstrip("?")
        off = 2 if name in FOURS else 4 if name in ("rng", "out") else 8
        _message(lib, call(lib, **{name: place[name] + off}), ALIGN, "aligned")


@pytest.mark.parametrize("call", [_forward, _backward])
def test_numbers_of_attention_are_looked_at(lib, call):
    inf, nan = float("inf"), float("nan")
    for bad in (0.0, -1.0, inf, nan):
        _message(lib, call(lib, scale=bad), INVALID, "scale must be positive and finite")
    for bad in (-1.0, inf, nan):
        _message(lib, call(lib, cap=bad), INVALID, "softcap must be >= 0 and finite")
    for bad in (dict(scale=2e30), dict(cap=2e30), dict(scale=1.0, cap=1e-38)):
        _message(lib, call(lib, **bad), INVALID, "at most 1e30")
    _message(lib, call(lib, dt=F32), DTYPE, "bf16")
    for bad in (dict(heads=0), dict(kv=0), dict(b=-1), dict(s=-1)):
        _message(lib, call(lib, **bad), SHAPE, "need b, s >= 0")
    _message(lib, call(lib, kv=3), SHAPE, "multiple of kv_heads")
    for hd in (0, 4, 60, 136):
        _message(lib, call(lib, hd=hd), SHAPE, "head_dim must be a multiple of 8")
    _message(lib, call(lib, b=1 << 16, s=1 << 16), SHAPE, "2^31-1")
    _message(lib, call(lib, b=1, s=(1 << 30) + 1), SHAPE, "2^30")
    _message(lib, call(lib, b=65536, s=1), SHAPE, "at most 65535")
    strides = call.__defaults__[call.__code__.co_varnames[1:].index("st")]
    for n in range(len(strides)):
        for bad in (0, -64, 68, 1 << 50):
            _message(lib, call(lib, st=strides[:n] + (bad,) + strides[n + 1:]), SHAPE, "strides must be positive multiples of 8")
    for n in ((6, 7) if call is _forward else range(8, 14)):
        _message(lib, call(lib, st=strides[:n] + (56 if n % 2 else strides[n] // 2,) + strides[n + 1:]), SHAPE, "heads overlap")


@pytest.mark.parametrize("call", [_rope, _rope_backward])
def test_numbers_of_the_norm_are_looked_at(lib, call):
    for eps in (0.0, -1.0, float("nan")):
        _message(lib, call(lib, eps=eps), INVALID, "eps must be > 0")
    for style in (-1, 2):
        _message(lib, call(lib, style=style), INVALID, "unknown rope style")
    _message(lib, call(lib, dt=3), DTYPE, "unsupported dtype")
    for rot in (0, 63, 66, -2):
        _message(lib, call(lib, rot=rot), SHAPE, "rot_dim must be even")
    for hd in (0, 60, 264):
        _message(lib, call(lib, hd=hd), SHAPE, "head_dim must be a multiple of 8")
    _message(lib, call(lib, table=0), SHAPE, "table_len must be >= 1")
    _message(lib, call(lib, heads=0), SHAPE, "need b, s >= 0")
    _message(lib, call(lib, heads=65537), SHAPE, "at most 65536 heads")
    strides = call.__defaults__[call.__code__.co_varnames[1:].index("st")]
    for n in range(len(strides)):
        for bad in (0, -64, 68, 1 << 50):
            _message(lib, call(lib, st=strides[:n] + (bad,) + strides[n + 1:]), SHAPE, "strides must be positive multiples of 8")
    for n in range(len(strides) - 4, len(strides)):
        _message(lib, call(lib, st=strides[:n] + (56 if n % 2 else strides[n] // 2,) + strides[n + 1:]), SHAPE, "heads overlap")


def test_numbers_of_key_ranges_are_looked_at(lib):
    for causal in (-1, 2):
        _message(lib, _ranges(lib, causal=causal), INVALID, "causal is 0 or 1")
    _message(lib, _ranges(lib, window=-1), INVALID, "window must be >= 0")
    _message(lib, _ranges(lib, causal=0), INVALID, "a prefix needs a causal mask")
    _message(lib, _ranges(lib, b=-1), SHAPE, "need b, s >= 0")
    _message(lib, _ranges(lib, b=1, s=(1 << 30) + 1), SHAPE, "2^30")


def test_workspaces_are_looked_at(lib):
    for call, size, name in ((_backward, lib.tpmlp_masked_attention_backward_workspace_size(2, 16, 4), "masked attention"),
                             (_rope_backward, lib.tpmlp_qk_norm_rope_backward_workspace_size(1, 8, 64), "qk_norm_rope")):
        _message(lib, call(lib, ws=None), WORKSPACE, name)
        _message(lib, call(lib, wsb=size - 1), WORKSPACE, name)
        _message(lib, call(lib, ws=AT[13] + 8), ALIGN, "workspace not")


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


def _cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("message,change", [
    ("key_range must be a contiguous torch.int32", dict(key_range=_cpu(1, 8, 2, dtype=torch.int64))),
    ("key_range must be a contiguous torch.int32", dict(key_range=_cpu(1, 4, 2, dtype=torch.int32))),
    ("key_range must be a contiguous torch.int32", dict(key_range=_cpu(1, 8, 4, dtype=torch.int32)[..., :2])),
    ("slopes must be a contiguous torch.float32", dict(slopes=torch.zeros(3))),
    ("slopes must be a contiguous torch.float32", dict(slopes=torch.zeros(2, dtype=torch.float64))),
    (r"k must be \[1, 8, 1, 64\]", dict(k=_cpu(1, 7, 1, 64))),
    (r"v must be \[1, 8, 1, 64\]", dict(v=_cpu(1, 8, 2, 64))),
    ("k must be torch.bfloat16", dict(k=_cpu(1, 8, 1, 64, dtype=torch.float32))),
    ("v must be torch.bfloat16", dict(v=_cpu(1, 8, 1, 64, dtype=torch.float16))),
    ("q needs contiguous columns", dict(q=_cpu(1, 8, 64, 2).transpose(2, 3))),
    ("must be CUDA tensors", {}),
])
def test_python_attention_names_what_it_refuses(message, change):
    args = dict(q=_cpu(1, 8, 2, 64), k=_cpu(1, 8, 1, 64), v=_cpu(1, 8, 1, 64), key_range=_cpu(1, 8, 2, dtype=torch.int32))
    args.update(change)
    with pytest.raises(ValueError, match=message):
        tp.masked_attention_forward(**args)
    grads = dict(o=_cpu(1, 8, 2, 64), lse=torch.zeros(1, 2, 8), do=_cpu(1, 8, 2, 64))
    with pytest.raises(ValueError, match=message):
        tp.masked_attention_backward(**args, **grads)


@pytest.mark.parametrize("message,change", [
    ("lse must be a contiguous torch.float32", dict(lse=torch.zeros(1, 8, 2))),
    ("lse must be a contiguous torch.float32", dict(lse=torch.zeros(1, 2, 8, dtype=torch.float64))),
    (r"o must be \[1, 8, 2, 64\]", dict(o=_cpu(1, 8, 2, 32))),
    ("o must be torch.bfloat16", dict(o=torch.zeros(1, 8, 2, 64))),
    (r"do must be \[1, 8, 2, 64\]", dict(do=_cpu(2, 8, 2, 64))),
    ("do must have o's strides", dict(do=_cpu(1, 8, 2, 128)[..., :64])),
])
def test_python_attention_backward_names_what_it_refuses(message, change):
    args = dict(o=_cpu(1, 8, 2, 64), lse=torch.zeros(1, 2, 8), do=_cpu(1, 8, 2, 64))
    args.update(change)
    with pytest.raises(ValueError, match=message):
        tp.masked_attention_backward(_cpu(1, 8, 2, 64), _cpu(1, 8, 1, 64), _cpu(1, 8, 1, 64), _cpu(1, 8, 2, dtype=torch.int32),
                                     **args)


def test_python_attention_names_strides_it_cannot_take():
    t, r = _cpu(2, 2, 8, 64).transpose(1, 2), _cpu(2, 8, 2, dtype=torch.int32)      # [b, heads, s, hd] memory
    with pytest.raises(ValueError, match="q needs contiguous columns and one stride for all tokens"):
        tp.masked_attention_forward(t, t, t, r)
    q = _cpu(2, 8, 2, 64)
    with pytest.raises(ValueError, match="k needs contiguous columns and one stride for all tokens"):
        tp.masked_attention_forward(q, t, t, r)
    with pytest.raises(ValueError, match="v needs contiguous columns and one stride for all tokens"):
        tp.masked_attention_forward(q, q, _cpu(2, 9, 2, 64)[:, 1:], r)              # a slice of the tokens


@pytest.mark.parametrize("message,change", [
    (r"cos and sin must be \[table_len, rot_dim / 2\]", dict(cos=torch.ones(64), sin=torch.ones(64))),
    ("sin must be a contiguous torch.float32", dict(sin=torch.ones(16, 31))),
    ("cos must be a contiguous torch.float32", dict(cos=torch.ones(16, 32, dtype=torch.float64))),
    ("gamma_q must be a contiguous torch.float32", dict(gamma_q=torch.ones(32))),
    ("gamma_k must be a contiguous torch.float32", dict(gamma_k=torch.ones(64, dtype=torch.bfloat16))),
    ("positions must be a contiguous torch.int32", dict(positions=torch.zeros(1, 8, dtype=torch.int64))),
    ("positions must be a contiguous torch.int32", dict(positions=torch.zeros(8, dtype=torch.int32))),
    (r"k must be \[1, 8, 1, 64\]", dict(k=_cpu(1, 8, 1, 32))),
    ("k must be torch.bfloat16", dict(k=torch.zeros(1, 8, 1, 64))),
    ("q needs contiguous columns", dict(q=_cpu(1, 8, 64, 2).transpose(2, 3))),
    ("must be CUDA tensors", {}),
])
def test_python_norm_names_what_it_refuses(message, change):
    args = dict(q=_cpu(1, 8, 2, 64), k=_cpu(1, 8, 1, 64), gamma_q=torch.ones(64), gamma_k=torch.ones(64),
                cos=torch.ones(16, 32), sin=torch.ones(16, 32))
    args.update(change)
    with pytest.raises(ValueError, match=message):
        tp.qk_norm_rope(**args)
    with pytest.raises(ValueError, match=message):
        tp.qk_norm_rope_backward(**args, dq_out=_cpu(1, 8, 2, 64), dk_out=_cpu(1, 8, 1, 64))


@pytest.mark.parametrize("message,change", [
    ("doc_ids must be a contiguous torch.int32", dict(doc_ids=torch.zeros(1, 7, dtype=torch.int32))),
    ("doc_ids must be a contiguous torch.int32", dict(doc_ids=torch.zeros(1, 8, dtype=torch.int64))),
    ("prefix_len must be a contiguous torch.int32", dict(prefix_len=torch.zeros(2, dtype=torch.int32))),
    ("must be CUDA tensors", dict(device="cpu")),
])
def test_python_key_ranges_name_what_they_refuse(message, change):
    with pytest.raises(ValueError, match=message):
        tp.attention_key_ranges(1, 8, **change)
