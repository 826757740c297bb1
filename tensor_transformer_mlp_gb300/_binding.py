"""Thin ctypes binding over libtpmlp.so (argument marshalling only).

Each function takes torch CUDA tensors, checks that their shapes and dtypes agree
with one another, and passes raw device pointers, sizes and the current CUDA
stream to the C entry point of the same name. Every step of the computation runs
in the library's kernels; if the library cannot be loaded, every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

from . import _build

GELU = {"erf": 0, "tanh": 1}
DTYPE = {torch.float32: 0, torch.bfloat16: 1}
RS_MODE = {"fused": 0, "splitk": 1}
GATE_ACT = {"gelu_erf": 0, "gelu_tanh": 1, "silu": 2}
WGRAD = {"f32": 0, "f32_add": 1, "operand": 2}
ROPE_STYLE = {"half": 0, "interleaved": 1}
STATUS = {0: "TPMLP_OK", 1: "TPMLP_ERR_INVALID", 2: "TPMLP_ERR_SHAPE", 3: "TPMLP_ERR_DTYPE", 4: "TPMLP_ERR_ALIGN",
          5: "TPMLP_ERR_CUDA", 6: "TPMLP_ERR_TIMEOUT", 7: "TPMLP_ERR_WORKSPACE"}

# Every entry point declared in include/tpmlp.h, with its ctypes signature.
_P, _I64, _I, _F, _U64, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_uint64, ctypes.c_size_t
_D = ctypes.c_double
SIGNATURES = {
    "tpmlp_forward": (_I, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _I, _I, _P]),
    "tpmlp_forward_biased": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _I, _I, _P]),
    "tpmlp_backward_workspace_size": (_SZ, [_I64, _I64, _I]),
    "tpmlp_backward_accumulate": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _I, _I, _P, _SZ, _P]),
    "tpmlp_backward_biased_workspace_size": (_SZ, [_I64, _I64, _I64, _I]),
    "tpmlp_backward_biased": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _I, _I, _P, _SZ,
                                   _P]),
    "tpmlp_backward": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _I, _I, _P, _SZ, _P]),
    "tpmlp_backward_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _I, _I, _P]),
    "tpmlp_sp_block_workspace_size": (_SZ, [_I64, _I64, _I64, _I64, _I, _I, _I]),
    "tpmlp_sp_block": (_I, [_P, _P, _P, _F, _P, _P, _D, _U64, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I, _I, _I, _I,
                            _P, _SZ, _P]),
    "tpmlp_sp_block_backward_workspace_size": (_SZ, [_I64, _I64, _I64, _I64, _I, _I]),
    "tpmlp_sp_block_backward": (_I, [_P, _P, _P, _F, _P, _P, _D, _U64, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64,
                                     _I64, _I64, _I, _I, _I, _P, _SZ, _P]),
    "tpmlp_sp_layernorm": (_I, [_P, _P, _P, _F, _P, _I64, _I64, _I, _P]),
    "tpmlp_rmsnorm": (_I, [_P, _P, _F, _P, _I64, _I64, _I, _P]),
    "tpmlp_rmsnorm_backward_workspace_size": (_SZ, [_I64, _I64]),
    "tpmlp_rmsnorm_backward": (_I, [_P, _P, _F, _P, _P, _P, _I64, _I64, _I, _P, _SZ, _P]),
    "tpmlp_sp_layernorm_backward_workspace_size": (_SZ, [_I64, _I64]),
    "tpmlp_sp_layernorm_backward": (_I, [_P, _P, _F, _P, _P, _P, _P, _P, _I64, _I64, _I, _P, _SZ, _P]),
    "tpmlp_sp_dropout_grad_gather": (_I, [_P, _P, _P, _D, _U64, _I64, _I64, _I64, _I, _I, _P]),
    "tpmlp_sp_gather": (_I, [_P, _P, _I64, _I64, _I64, _I, _I, _P]),
    "tpmlp_sp_reduce_scatter": (_I, [_P, _P, _I64, _I64, _I64, _I, _I, _P]),
    "tpmlp_sp_dropout_residual": (_I, [_P, _P, _P, _P, _D, _U64, _I64, _I64, _I64, _I, _I, _P]),
    "tpmlp_attention_forward_workspace_size": (_SZ, [_I64, _I64, _I64, _I, _I]),
    "tpmlp_attention_forward": (_I, [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _I, _I, _P, _SZ, _P]),
    "tpmlp_attention_backward_workspace_size": (_SZ, [_I64, _I64, _I64, _I, _I]),
    "tpmlp_attention_backward": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _I, _I, _P, _SZ,
                                      _P]),
    "tpmlp_attention_key_ranges": (_I, [_P, _P, _I, _I64, _P, _I64, _I64, _P]),
    "tpmlp_qk_norm_rope": (_I, [_P, _P, _P, _P, _F, _P, _P, _P, _I64, _I, _I, _P, _P, _I64, _I64, _I, _I, _I]
                           + [_I64] * 8 + [_I, _P]),
    "tpmlp_qk_norm_rope_backward_workspace_size": (_SZ, [_I64, _I64, _I]),
    "tpmlp_qk_norm_rope_backward": (_I, [_P, _P, _P, _P, _F, _P, _P, _P, _I64, _I, _I, _P, _P, _P, _P, _P, _P, _I64,
                                         _I64, _I, _I, _I] + [_I64] * 12 + [_I, _P, _SZ, _P]),
    "tpmlp_masked_attention_forward": (_I, [_P, _P, _P, _P, _P, _F, _F, _P, _P, _I64, _I64, _I, _I, _I] + [_I64] * 8
                                       + [_I, _P]),
    "tpmlp_masked_attention_backward_workspace_size": (_SZ, [_I64, _I64, _I]),
    "tpmlp_masked_attention_backward": (_I, [_P, _P, _P, _P, _P, _F, _F, _P, _P, _P, _P, _P, _P, _I64, _I64, _I, _I, _I]
                                        + [_I64] * 14 + [_I, _P, _SZ, _P]),
    "tpmlp_gated_forward_workspace_size": (_SZ, [_I64, _I64, _I64, _I, _I]),
    "tpmlp_gated_forward": (_I, [_P] * 6 + [_I64, _I64, _I64, _I, _I, _I, _P, _SZ, _P]),
    "tpmlp_gated_backward_workspace_size": (_SZ, [_I64, _I64, _I64, _I]),
    "tpmlp_gated_backward": (_I, [_P] * 9 + [_I64, _I64, _I64, _I, _I, _I, _I, _P, _SZ, _P]),
    "tpmlp_residual_norm": (_I, [_P] * 5 + [_F, _F, _P, _P, _I64, _I64, _I64, _I, _P]),
    "tpmlp_residual_norm_backward_workspace_size": (_SZ, [_I64, _I64, _I64, _I]),
    "tpmlp_residual_norm_backward": (_I, [_P] * 7 + [_F, _F] + [_P] * 5 + [_I64, _I64, _I64, _I, _P, _SZ, _P]),
    "tpmlp_last_error": (ctypes.c_char_p, []),
    "tpmlp_device_status": (_I, [_P, _I]),
    "tpmlp_check_wait_timeout": (_I, [_U64, _P]),
    "tpmlp_set_gemm_variant": (_I, [_I, _I, _I]),
}

_lib = None
_lock = threading.Lock()


class TpmlpError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


def load_library(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load (building first if it is missing or stale) libtpmlp.so and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if build_if_missing and _build.is_stale():
                _build.build()
            if not os.path.exists(_build.LIB_PATH):
                raise RuntimeError(f"libtpmlp.so is missing at {_build.LIB_PATH}; run the build first")
            lib = ctypes.CDLL(_build.LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def _check(status: int) -> None:
    if status != 0:
        msg = load_library().tpmlp_last_error().decode(errors="replace")
        raise TpmlpError(status, msg)


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _cuda(*ts: torch.Tensor | None) -> None:
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


class _On:
    """Makes a device and a stream current for a while, so that what torch allocates meanwhile belongs to that stream."""
    __slots__ = ("guard",)

    def __init__(self, index: int, stream):
        # torch.cuda.stream switches to the stream's device too
        self.guard = torch.cuda.device(index) if stream is None else torch.cuda.stream(stream)

    def __enter__(self):
        self.guard.__enter__()

    def __exit__(self, *exc):
        self.guard.__exit__(*exc)
        return False


_HERE = contextlib.nullcontext()


def _where(index: int, stream):
    """A context in which the device `index` and `stream` (default: the device's current stream) are current, and the
    stream's handle. Where both are current already there is nothing to switch."""
    if index < 0:
        raise ValueError("tensors must be CUDA tensors")
    if stream is None:
        here = _HERE if torch._C._cuda_getDevice() == index else _On(index, None)
        return here, torch._C._cuda_getCurrentRawStream(index)
    if stream.device_index != index:
        raise ValueError(f"the stream is on cuda:{stream.device_index}, the tensors are on cuda:{index}")
    return _On(index, stream), stream.cuda_stream


def _device(first: torch.Tensor, *rest: torch.Tensor | None) -> int:
    """The index of the one device that all tensors are on (-1: the CPU)."""
    index = first.get_device()
    for t in rest:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors are on different devices ({first.device}, {t.device})")
    return index


def _heads(t: torch.Tensor, shape: tuple[int, int, int, int], dtype: torch.dtype, name: str) -> tuple[int, int]:
    """The (token, head) strides of a [b, s, heads, hd] tensor of heads."""
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    b, s, heads, hd = shape
    sb, ss, sh, sc = t.stride()
    if (sc != 1 and hd > 1) or (b > 1 and s > 1 and sb != s * ss):
        raise ValueError(f"{name} needs contiguous columns and one stride for all tokens of the batch")
    return ss if s > 1 else sb if b > 1 else max(heads * hd, 8), sh if heads > 1 else hd


def _out(t, shape: tuple[int, int, int, int], like: torch.Tensor, name: str):
    """The output `t`, or a new contiguous one of like's type, and its (token, head) strides."""
    if t is None:
        return torch.empty(shape, dtype=like.dtype, device=like.device), (shape[2] * shape[3], shape[3])
    return t, _heads(t, shape, like.dtype, name)


def _dense(t: torch.Tensor, shape: tuple[int, ...], dtype: torch.dtype, name: str) -> None:
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)}")


def _dt(t: torch.Tensor) -> int:
    if t.dtype not in DTYPE:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return DTYPE[t.dtype]


# ----------------------------------------------------------------------- C-ABI mirrors

def tpmlp_forward(X, A, B, O, Z_save, Y_save, t: int, gelu: str = "tanh", stream=None) -> None:
    n, d = X.shape
    m = A.shape[1]
    assert A.shape == (d, m) and B.shape == (m, d) and O.shape == (n, d) and Y_save.shape == (n, m)
    assert Z_save is None or Z_save.shape == (n, m)
    _cuda(X, A, B, O, Z_save, Y_save)
    _check(load_library().tpmlp_forward(_ptr(X), _ptr(A), _ptr(B), _ptr(O), _ptr(Z_save), _ptr(Y_save), n, d, m, t,
                                        GELU[gelu], _dt(X), _stream(stream)))


def tpmlp_forward_biased(X, A, B, bias1, bias2, O, Z_save, Y_save, t: int, gelu: str = "tanh", stream=None) -> None:
    n, d = X.shape
    m = A.shape[1]
    assert A.shape == (d, m) and B.shape == (m, d) and O.shape == (n, d) and Y_save.shape == (n, m)
    assert bias1.shape == (m,) and bias2.shape == (d,) and bias1.dtype == X.dtype and bias2.dtype == X.dtype
    assert Z_save is None or Z_save.shape == (n, m)
    _cuda(X, A, B, bias1, bias2, O, Z_save, Y_save)
    _check(load_library().tpmlp_forward_biased(_ptr(X), _ptr(A), _ptr(B), _ptr(bias1), _ptr(bias2), _ptr(O),
                                               _ptr(Z_save), _ptr(Y_save), n, d, m, t, GELU[gelu], _dt(X),
                                               _stream(stream)))


def tpmlp_backward_accumulate(X, A, B, G, Z_save, Y_save, dX, dA, dB, t: int, gelu: str = "tanh", workspace=None,
                              stream=None) -> None:
    """tpmlp_backward, but dA += X^T D and dB += Y^T G into the given fp32 buffers."""
    n, d = X.shape
    m = A.shape[1]
    assert G.shape == (n, d) and Z_save.shape == (n, m) and Y_save.shape == (n, m) and dX.shape == (n, d)
    assert dA.shape == (d, m) and dB.shape == (m, d) and dA.dtype == torch.float32 and dB.dtype == torch.float32
    _cuda(X, A, B, G, Z_save, Y_save, dX, dA, dB, workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().tpmlp_backward_accumulate(_ptr(X), _ptr(A), _ptr(B), _ptr(G), _ptr(Z_save), _ptr(Y_save),
                                                    _ptr(dX), _ptr(dA), _ptr(dB), n, d, m, t, GELU[gelu], _dt(X),
                                                    _ptr(workspace), ws_bytes, _stream(stream)))


def tpmlp_backward_biased_workspace_size(n: int, d: int, m: int, dtype: torch.dtype) -> int:
    return load_library().tpmlp_backward_biased_workspace_size(n, d, m, DTYPE[dtype])


def tpmlp_backward_biased(X, A, B, G, Z_save, Y_save, dX, dA, dB, dbias1, dbias2, t: int, gelu: str = "tanh",
                          workspace=None, stream=None) -> None:
    n, d = X.shape
    m = A.shape[1]
    assert G.shape == (n, d) and Z_save.shape == (n, m) and Y_save.shape == (n, m) and dX.shape == (n, d)
    assert dA.shape == (d, m) and dB.shape == (m, d) and dbias1.shape == (m,) and dbias2.shape == (d,)
    for g_ in (dA, dB, dbias1, dbias2):
        assert g_.dtype == torch.float32
    _cuda(X, A, B, G, Z_save, Y_save, dX, dA, dB, dbias1, dbias2, workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().tpmlp_backward_biased(_ptr(X), _ptr(A), _ptr(B), _ptr(G), _ptr(Z_save), _ptr(Y_save),
                                                _ptr(dX), _ptr(dA), _ptr(dB), _ptr(dbias1), _ptr(dbias2), n, d, m, t,
                                                GELU[gelu], _dt(X), _ptr(workspace), ws_bytes, _stream(stream)))


def tpmlp_backward_workspace_size(n: int, m: int, dtype: torch.dtype) -> int:
    return load_library().tpmlp_backward_workspace_size(n, m, DTYPE[dtype])


def tpmlp_backward(X, A, B, G, Z_save, Y_save, dX, dA, dB, t: int, gelu: str = "tanh", workspace=None,
                   stream=None) -> None:
    n, d = X.shape
    m = A.shape[1]
    assert G.shape == (n, d) and Z_save.shape == (n, m) and Y_save.shape == (n, m) and dX.shape == (n, d)
    assert dA.shape == (d, m) and dB.shape == (m, d) and dA.dtype == torch.float32 and dB.dtype == torch.float32
    _cuda(X, A, B, G, Z_save, Y_save, dX, dA, dB, workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().tpmlp_backward(_ptr(X), _ptr(A), _ptr(B), _ptr(G), _ptr(Z_save), _ptr(Y_save), _ptr(dX),
                                         _ptr(dA), _ptr(dB), n, d, m, t, GELU[gelu], _dt(X), _ptr(workspace),
                                         ws_bytes, _stream(stream)))


def tpmlp_sp_block_workspace_size(b, s, h, m, t, dtype: torch.dtype, rs: str = "fused") -> int:
    return load_library().tpmlp_sp_block_workspace_size(b, s, h, m, t, DTYPE[dtype], RS_MODE[rs])


def tpmlp_sp_block(x_shards, gamma, beta, eps, A, B, p_drop, seed, out_shards, mask_bits, t: int, gelu="tanh",
                   rs="fused", workspace=None, stream=None, Z_save=None, Y_save=None) -> None:
    tt, b, sl, h = x_shards.shape
    assert tt == t and out_shards.shape == x_shards.shape
    m = A.shape[1]
    assert A.shape == (h, m) and B.shape == (m, h) and gamma.shape == (h,) and beta.shape == (h,)
    assert gamma.dtype == torch.float32 and beta.dtype == torch.float32
    if mask_bits is not None:
        assert mask_bits.dtype in (torch.int32, torch.uint32) and mask_bits.numel() >= (b * sl * t * h + 31) // 32
    for sv in (Z_save, Y_save):
        assert sv is None or sv.shape == (b * sl * t, m)
    _cuda(x_shards, gamma, beta, A, B, out_shards, mask_bits, workspace, Z_save, Y_save)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().tpmlp_sp_block(_ptr(x_shards), _ptr(gamma), _ptr(beta), eps, _ptr(A), _ptr(B), p_drop,
                                         seed, _ptr(out_shards), _ptr(mask_bits), _ptr(Z_save), _ptr(Y_save), b,
                                         sl * t, h, m, t, GELU[gelu], _dt(x_shards), RS_MODE[rs], _ptr(workspace),
                                         ws_bytes, _stream(stream)))


def tpmlp_sp_block_backward_workspace_size(b, s, h, m, t, dtype: torch.dtype) -> int:
    return load_library().tpmlp_sp_block_backward_workspace_size(b, s, h, m, t, DTYPE[dtype])


def tpmlp_sp_block_backward(x_shards, gamma, beta, eps, A, B, p_drop, seed, Z_save, Y_save, dout_shards, dx_shards,
                            dgamma, dbeta, dA, dB, t: int, gelu="tanh", workspace=None, stream=None,
                            mask_bits=None) -> None:
    tt, b, sl, h = x_shards.shape
    m = A.shape[1]
    assert tt == t and dout_shards.shape == x_shards.shape and dx_shards.shape == x_shards.shape
    assert Z_save.shape == (b * sl * t, m) and Y_save.shape == (b * sl * t, m)
    assert dgamma.shape == (h,) and dbeta.shape == (h,) and dA.shape == (h, m) and dB.shape == (m, h)
    assert mask_bits is None or mask_bits.numel() * 32 >= x_shards.numel()
    _cuda(x_shards, gamma, beta, A, B, Z_save, Y_save, dout_shards, dx_shards, dgamma, dbeta, dA, dB, workspace,
          mask_bits)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().tpmlp_sp_block_backward(
        _ptr(x_shards), _ptr(gamma), _ptr(beta), eps, _ptr(A), _ptr(B), p_drop, seed, _ptr(mask_bits), _ptr(Z_save),
        _ptr(Y_save),
        _ptr(dout_shards), _ptr(dx_shards), _ptr(dgamma), _ptr(dbeta), _ptr(dA), _ptr(dB), b, sl * t, h, m, t,
        GELU[gelu], _dt(x_shards), _ptr(workspace), ws_bytes, _stream(stream)))


def tpmlp_sp_layernorm(x, gamma, beta, eps, y, stream=None) -> None:
    h = x.shape[-1]
    rows = x.numel() // h
    assert y.shape == x.shape and gamma.shape == (h,) and beta.shape == (h,)
    _cuda(x, gamma, beta, y)
    _check(load_library().tpmlp_sp_layernorm(_ptr(x), _ptr(gamma), _ptr(beta), eps, _ptr(y), rows, h, _dt(x),
                                             _stream(stream)))


def tpmlp_rmsnorm(x, gamma, eps, y, stream=None) -> None:
    h = x.shape[-1]
    rows = x.numel() // h
    assert y.shape == x.shape and gamma.shape == (h,) and gamma.dtype == torch.float32
    _cuda(x, gamma, y)
    _check(load_library().tpmlp_rmsnorm(_ptr(x), _ptr(gamma), eps, _ptr(y), rows, h, _dt(x), _stream(stream)))


def tpmlp_rmsnorm_backward_workspace_size(rows: int, h: int) -> int:
    return load_library().tpmlp_rmsnorm_backward_workspace_size(rows, h)


def tpmlp_rmsnorm_backward(x, gamma, eps, dy, dx, dgamma, workspace, stream=None) -> None:
    h = x.shape[-1]
    rows = x.numel() // h
    assert dy.shape == x.shape and dx.shape == x.shape and gamma.shape == (h,) and dgamma.shape == (h,)
    assert dgamma.dtype == torch.float32 and workspace.dtype == torch.uint8
    _cuda(x, gamma, dy, dx, dgamma, workspace)
    _check(load_library().tpmlp_rmsnorm_backward(_ptr(x), _ptr(gamma), eps, _ptr(dy), _ptr(dx), _ptr(dgamma), rows, h,
                                                 _dt(x), _ptr(workspace), workspace.numel(), _stream(stream)))


def tpmlp_sp_layernorm_backward_workspace_size(rows: int, h: int) -> int:
    return load_library().tpmlp_sp_layernorm_backward_workspace_size(rows, h)


def tpmlp_sp_layernorm_backward(x, gamma, eps, dy, dres, dx, dgamma, dbeta, workspace, stream=None) -> None:
    h = x.shape[-1]
    rows = x.numel() // h
    assert dy.shape == x.shape and dx.shape == x.shape and gamma.shape == (h,)
    assert dres is None or (dres.shape == x.shape and dres.dtype == x.dtype)
    assert dgamma.shape == (h,) and dbeta.shape == (h,) and dgamma.dtype == dbeta.dtype == torch.float32
    assert workspace.dtype == torch.uint8
    _cuda(x, gamma, dy, dres, dx, dgamma, dbeta, workspace)
    _check(load_library().tpmlp_sp_layernorm_backward(_ptr(x), _ptr(gamma), eps, _ptr(dy), _ptr(dres), _ptr(dx),
                                                      _ptr(dgamma), _ptr(dbeta), rows, h, _dt(x), _ptr(workspace),
                                                      workspace.numel(), _stream(stream)))


def tpmlp_sp_dropout_grad_gather(dout_shards, dtok, p_drop: float, seed: int, stream=None, mask_bits=None) -> None:
    t, b, sl, h = dout_shards.shape
    assert dtok.shape == (b, sl * t, h) and dtok.dtype == dout_shards.dtype
    assert mask_bits is None or mask_bits.numel() * 32 >= dout_shards.numel()
    _cuda(dout_shards, dtok, mask_bits)
    _check(load_library().tpmlp_sp_dropout_grad_gather(_ptr(dout_shards), _ptr(dtok), _ptr(mask_bits), float(p_drop),
                                                       seed, b, sl * t, h, t, _dt(dout_shards), _stream(stream)))


def tpmlp_sp_gather(x_shards, x_full, stream=None) -> None:
    t, b, sl, h = x_shards.shape
    assert x_full.shape == (b, sl * t, h) and x_full.dtype == x_shards.dtype
    _cuda(x_shards, x_full)
    _check(load_library().tpmlp_sp_gather(_ptr(x_shards), _ptr(x_full), b, sl * t, h, t, _dt(x_shards),
                                          _stream(stream)))


def tpmlp_sp_reduce_scatter(partials, out_shards, stream=None) -> None:
    t, b, sl, h = out_shards.shape
    assert partials.shape == (t, b * sl * t, h) and partials.dtype == torch.float32
    _cuda(partials, out_shards)
    _check(load_library().tpmlp_sp_reduce_scatter(_ptr(partials), _ptr(out_shards), b, sl * t, h, t,
                                                  _dt(out_shards), _stream(stream)))


def tpmlp_sp_dropout_residual(x_shards, y_shards, out_shards, mask_bits, p_drop, seed, stream=None) -> None:
    t, b, sl, h = x_shards.shape
    assert y_shards.shape == x_shards.shape and out_shards.shape == x_shards.shape
    _cuda(x_shards, y_shards, out_shards, mask_bits)
    _check(load_library().tpmlp_sp_dropout_residual(_ptr(x_shards), _ptr(y_shards), _ptr(out_shards),
                                                    _ptr(mask_bits), p_drop, seed, b, sl * t, h, t, _dt(x_shards),
                                                    _stream(stream)))


def tpmlp_check_wait_timeout(limit_ns: int, stream=None) -> None:
    _check(load_library().tpmlp_check_wait_timeout(limit_ns, _stream(stream)))


def tpmlp_device_status(stream=None, clear: bool = True) -> None:
    _check(load_library().tpmlp_device_status(_stream(stream), 1 if clear else 0))


def tpmlp_set_gemm_variant(pair_kernel: int = 1, pair_pacing: int = 1, pair_group: int = 0) -> None:
    _check(load_library().tpmlp_set_gemm_variant(pair_kernel, pair_pacing, pair_group))


# ----------------------------------------------------------------------- conveniences

def forward(X, A, B, t: int, gelu: str = "tanh", save_z: bool = True, stream=None, bias1=None, bias2=None):
    """Allocate O, Z, Y with torch and run tpmlp_forward (tpmlp_forward_biased when biases are
    given). Returns (O, Z, Y)."""
    n, m = X.shape[0], A.shape[1]
    O = torch.empty_like(X)
    Z = torch.empty((n, m), dtype=X.dtype, device=X.device) if save_z else None
    Y = torch.empty((n, m), dtype=X.dtype, device=X.device)
    if bias1 is not None or bias2 is not None:
        tpmlp_forward_biased(X, A, B, bias1, bias2, O, Z, Y, t, gelu, stream)
    else:
        tpmlp_forward(X, A, B, O, Z, Y, t, gelu, stream)
    return O, Z, Y


def backward(X, A, B, G, Z, Y, t: int, gelu: str = "tanh", stream=None, with_bias: bool = False):
    """Allocate gradients and the workspace with torch and run tpmlp_backward (or, with_bias,
    tpmlp_backward_biased). Returns (dX, dA, dB) or (dX, dA, dB, dbias1, dbias2)."""
    n, d = X.shape
    m = A.shape[1]
    dX = torch.empty_like(X)
    dA = torch.empty((d, m), dtype=torch.float32, device=X.device)
    dB = torch.empty((m, d), dtype=torch.float32, device=X.device)
    if with_bias:
        db1 = torch.empty(m, dtype=torch.float32, device=X.device)
        db2 = torch.empty(d, dtype=torch.float32, device=X.device)
        ws = torch.empty(max(1, tpmlp_backward_biased_workspace_size(n, d, m, X.dtype)), dtype=torch.uint8,
                         device=X.device)
        tpmlp_backward_biased(X, A, B, G, Z, Y, dX, dA, dB, db1, db2, t, gelu, ws, stream)
        return dX, dA, dB, db1, db2
    ws = torch.empty(max(1, tpmlp_backward_workspace_size(n, m, X.dtype)), dtype=torch.uint8, device=X.device)
    tpmlp_backward(X, A, B, G, Z, Y, dX, dA, dB, t, gelu, ws, stream)
    return dX, dA, dB


def sp_block(x_shards, gamma, beta, eps, A, B, p_drop, seed, t: int, gelu="tanh", rs="fused", with_mask=True,
             save_for_backward=False, stream=None):
    """Allocate outputs and workspace and run tpmlp_sp_block.
    Returns (out_shards, mask_bits or None, (Z, Y) or None)."""
    tt, b, sl, h = x_shards.shape
    n, m = b * sl * t, A.shape[1]
    out = torch.empty_like(x_shards)
    mask = torch.empty(((n * h + 31) // 32,), dtype=torch.int32, device=x_shards.device) if with_mask else None
    saves = None
    if save_for_backward:
        saves = tuple(torch.empty((n, m), dtype=x_shards.dtype, device=x_shards.device) for _ in range(2))
    ws = torch.empty(max(1, tpmlp_sp_block_workspace_size(b, sl * t, h, m, t, x_shards.dtype, rs)),
                     dtype=torch.uint8, device=x_shards.device)
    tpmlp_sp_block(x_shards, gamma, beta, eps, A, B, p_drop, seed, out, mask, t, gelu, rs, ws, stream,
                   *(saves if saves else (None, None)))
    return out, mask, saves


def sp_block_backward(x_shards, gamma, beta, eps, A, B, p_drop, seed, Z, Y, dout_shards, t: int, gelu="tanh",
                      stream=None, mask_bits=None):
    """Allocate gradients and workspace and run tpmlp_sp_block_backward.
    Returns (dx_shards, dgamma, dbeta, dA, dB)."""
    tt, b, sl, h = x_shards.shape
    m = A.shape[1]
    dev = x_shards.device
    dx = torch.empty_like(x_shards)
    dgamma = torch.empty(h, dtype=torch.float32, device=dev)
    dbeta = torch.empty(h, dtype=torch.float32, device=dev)
    dA = torch.empty((h, m), dtype=torch.float32, device=dev)
    dB = torch.empty((m, h), dtype=torch.float32, device=dev)
    ws = torch.empty(max(1, tpmlp_sp_block_backward_workspace_size(b, sl * t, h, m, t, x_shards.dtype)),
                     dtype=torch.uint8, device=dev)
    tpmlp_sp_block_backward(x_shards, gamma, beta, eps, A, B, p_drop, seed, Z, Y, dout_shards, dx, dgamma, dbeta, dA,
                            dB, t, gelu, ws, stream, mask_bits)
    return dx, dgamma, dbeta, dA, dB


# ----------------------------------------------------------------------- attention block

def rmsnorm(x, gamma, eps: float = 1e-5, stream=None):
    """Allocates y and runs tpmlp_rmsnorm."""
    y = torch.empty_like(x)
    tpmlp_rmsnorm(x, gamma, eps, y, stream)
    return y


def rmsnorm_backward(x, gamma, dy, eps: float = 1e-5, stream=None):
    """Allocates dx, dgamma and the workspace and runs tpmlp_rmsnorm_backward; returns (dx, dgamma)."""
    h = x.shape[-1]
    dx = torch.empty_like(x)
    dgamma = torch.empty(h, dtype=torch.float32, device=x.device)
    ws = torch.empty(tpmlp_rmsnorm_backward_workspace_size(x.numel() // h, h), dtype=torch.uint8, device=x.device)
    tpmlp_rmsnorm_backward(x, gamma, eps, dy, dx, dgamma, ws, stream)
    return dx, dgamma


def attention_forward(X, Wqkv, Wo, heads: int, t: int, stream=None):
    """X [b, s, h] bf16; allocates Y, the saves and the workspace and runs tpmlp_attention_forward.
    Returns (Y [b, s, h], (QKV, P, O))."""
    b, s, h = X.shape
    _cuda(X, Wqkv, Wo)
    assert Wqkv.shape == (h, 3 * h) and Wo.shape == (h, h)
    dev = X.device
    Y = torch.empty_like(X)
    QKV = torch.empty((b * s, 3 * h), dtype=X.dtype, device=dev)
    P = torch.empty((b, heads, s, s), dtype=X.dtype, device=dev)
    O = torch.empty((b * s, h), dtype=X.dtype, device=dev)
    lib = load_library()
    ws = torch.empty(max(1, lib.tpmlp_attention_forward_workspace_size(b, s, h, heads, _dt(X))), dtype=torch.uint8,
                     device=dev)
    _check(lib.tpmlp_attention_forward(_ptr(X), _ptr(Wqkv), _ptr(Wo), _ptr(Y), _ptr(QKV), _ptr(P), _ptr(O), b, s, h,
                                       heads, t, _dt(X), _ptr(ws), ws.numel(), _stream(stream)))
    return Y, (QKV, P, O)


def attention_backward(X, Wqkv, Wo, G, saves, heads: int, t: int, stream=None):
    """Runs tpmlp_attention_backward; returns (dX [b, s, h], dWqkv [h, 3h] fp32, dWo [h, h] fp32)."""
    b, s, h = X.shape
    QKV, P, O = saves
    _cuda(X, Wqkv, Wo, G, QKV, P, O)
    dev = X.device
    dX = torch.empty_like(X)
    dWqkv = torch.empty((h, 3 * h), dtype=torch.float32, device=dev)
    dWo = torch.empty((h, h), dtype=torch.float32, device=dev)
    lib = load_library()
    ws = torch.empty(max(1, lib.tpmlp_attention_backward_workspace_size(b, s, h, heads, _dt(X))), dtype=torch.uint8,
                     device=dev)
    _check(lib.tpmlp_attention_backward(_ptr(X), _ptr(Wqkv), _ptr(Wo), _ptr(G), _ptr(QKV), _ptr(P), _ptr(O), _ptr(dX),
                                        _ptr(dWqkv), _ptr(dWo), b, s, h, heads, t, _dt(X), _ptr(ws), ws.numel(),
                                        _stream(stream)))
    return dX, dWqkv, dWo


# ----------------------------------------------------------------------- masked attention

def attention_key_ranges(b: int, s: int, doc_ids=None, prefix_len=None, causal: bool = True, window: int = 0,
                         device=None, stream=None):
    """Runs tpmlp_attention_key_ranges; returns the int32 [b, s, 2] key range of every query, for
    masked_attention_forward and _backward. doc_ids int32 [b, s], prefix_len int32 [b]; `device` defaults to theirs,
    else to the current one."""
    if device is not None:
        device = torch.device(device)
    given = doc_ids if doc_ids is not None else prefix_len
    if doc_ids is not None:
        _dense(doc_ids, (b, s), torch.int32, "doc_ids")
    if given is not None:
        index = _device(given, prefix_len)
        if device is not None and (device.type != given.device.type or device.index not in (None, given.device.index)):
            raise ValueError(f"doc_ids or prefix_len are on {given.device}, not on {device}")
    else:
        device = torch.device("cuda") if device is None else device
        index = -1 if device.type != "cuda" else torch.cuda.current_device() if device.index is None else device.index
    if prefix_len is not None:
        _dense(prefix_len, (b,), torch.int32, "prefix_len")
    lib = load_library()
    here, st = _where(index, stream)
    with here:
        out = torch.empty((b, s, 2), dtype=torch.int32, device="cuda")
        _check(lib.tpmlp_attention_key_ranges(_ptr(doc_ids), _ptr(prefix_len), 1 if causal else 0, max(-1, min(window, s)),
                                              out.data_ptr(), b, s, st))  # a longer window hides nothing; -1: refused
    return out


def rope_tables(table_len: int, rot_dim: int, theta: float = 10000.0, device=None):
    """The fp32 (cos, sin) tables [table_len, rot_dim / 2] of the angles pos * theta^(-2i / rot_dim), computed in
    64 bits so that far positions keep their phase."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim must be even and at least 2, got {rot_dim}")
    inv = theta ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    ang = torch.arange(table_len, dtype=torch.float64, device=device)[:, None] * inv
    return ang.cos().float(), ang.sin().float()


def _rope_args(q, k, gamma_q, gamma_k, cos, sin, positions):
    b, s, heads, hd = shape = q.shape
    kshape = (b, s, k.shape[2], hd)
    table = cos.shape
    if len(table) != 2:
        raise ValueError("cos and sin must be [table_len, rot_dim / 2]")
    strides = _heads(q, shape, q.dtype, "q") + _heads(k, kshape, q.dtype, "k")
    _dense(gamma_q, (hd,), torch.float32, "gamma_q")
    _dense(gamma_k, (hd,), torch.float32, "gamma_k")
    _dense(cos, table, torch.float32, "cos")
    _dense(sin, table, torch.float32, "sin")
    if positions is not None:
        _dense(positions, (b, s), torch.int32, "positions")
    return shape, kshape, table[0], 2 * table[1], strides


def qk_norm_rope(q, k, gamma_q, gamma_k, cos, sin, eps: float = 1e-5, positions=None, style: str = "half",
                 q_out=None, k_out=None, stream=None):
    """q [b, s, heads, head_dim], k [b, s, kv_heads, head_dim] (views of a QKV matrix, for instance). Allocates
    q_out and k_out unless given (q and k themselves for in place) and runs tpmlp_qk_norm_rope; returns them."""
    shape, kshape, table_len, rot, strides = _rope_args(q, k, gamma_q, gamma_k, cos, sin, positions)
    lib = load_library()
    here, st = _where(_device(q, k, gamma_q, gamma_k, cos, sin, positions, q_out, k_out), stream)
    with here:
        q_out, sq = _out(q_out, shape, q, "q_out")
        k_out, sk = _out(k_out, kshape, q, "k_out")
        _check(lib.tpmlp_qk_norm_rope(
            q.data_ptr(), k.data_ptr(), gamma_q.data_ptr(), gamma_k.data_ptr(), eps, cos.data_ptr(), sin.data_ptr(),
            _ptr(positions), table_len, rot, ROPE_STYLE[style], q_out.data_ptr(), k_out.data_ptr(), shape[0], shape[1],
            shape[2], kshape[2], shape[3], *strides, *sq, *sk, _dt(q), st))
    return q_out, k_out


def qk_norm_rope_backward(q, k, gamma_q, gamma_k, cos, sin, dq_out, dk_out, eps: float = 1e-5, positions=None,
                          style: str = "half", dq=None, dk=None, stream=None):
    """Runs tpmlp_qk_norm_rope_backward from the gradients of q_out and k_out; allocates the workspace, the gains'
    gradients and, unless given, dq and dk. Returns (dq, dk, dgamma_q, dgamma_k)."""
    shape, kshape, table_len, rot, strides = _rope_args(q, k, gamma_q, gamma_k, cos, sin, positions)
    b, s, heads, hd = shape
    strides += _heads(dq_out, shape, q.dtype, "dq_out") + _heads(dk_out, kshape, q.dtype, "dk_out")
    lib = load_library()
    here, st = _where(_device(q, k, gamma_q, gamma_k, cos, sin, positions, dq_out, dk_out, dq, dk), stream)
    with here:
        device = q.device
        dq, sq = _out(dq, shape, q, "dq")
        dk, sk = _out(dk, kshape, q, "dk")
        dgq = torch.empty(hd, dtype=torch.float32, device=device)
        dgk = torch.empty(hd, dtype=torch.float32, device=device)
        ws_bytes = lib.tpmlp_qk_norm_rope_backward_workspace_size(b, s, hd)
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=device)
        _check(lib.tpmlp_qk_norm_rope_backward(
            q.data_ptr(), k.data_ptr(), gamma_q.data_ptr(), gamma_k.data_ptr(), eps, cos.data_ptr(), sin.data_ptr(),
            _ptr(positions), table_len, rot, ROPE_STYLE[style], dq_out.data_ptr(), dk_out.data_ptr(), dq.data_ptr(),
            dk.data_ptr(), dgq.data_ptr(), dgk.data_ptr(), b, s, heads, kshape[2], hd, *strides, *sq, *sk, _dt(q),
            ws.data_ptr(), ws_bytes, st))
    return dq, dk, dgq, dgk


def _masked_args(q, k, v, key_range, slopes):
    b, s, heads, hd = shape = q.shape
    kshape = (b, s, k.shape[2], hd)
    _dense(key_range, (b, s, 2), torch.int32, "key_range")
    if slopes is not None:
        _dense(slopes, (heads,), torch.float32, "slopes")
    dtype = q.dtype
    return shape, kshape, _heads(q, shape, dtype, "q") + _heads(k, kshape, dtype, "k") + _heads(v, kshape, dtype, "v")


def masked_attention_forward(q, k, v, key_range, scale: float | None = None, softcap: float = 0.0, slopes=None,
                             o=None, stream=None):
    """q [b, s, heads, head_dim], k and v [b, s, kv_heads, head_dim] bf16 (views of a QKV matrix, for instance).
    Allocates o (unless given) and lse and runs tpmlp_masked_attention_forward; scale defaults to
    head_dim^-1/2. Returns (o [b, s, heads, head_dim], lse [b, heads, s] fp32)."""
    shape, kshape, strides = _masked_args(q, k, v, key_range, slopes)
    b, s, heads, hd = shape
    lib = load_library()
    here, st = _where(_device(q, k, v, key_range, slopes, o), stream)
    with here:
        o, so = _out(o, shape, q, "o")
        lse = torch.empty((b, heads, s), dtype=torch.float32, device=q.device)
        _check(lib.tpmlp_masked_attention_forward(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), key_range.data_ptr(), _ptr(slopes),
            hd ** -0.5 if scale is None else scale, softcap, o.data_ptr(), lse.data_ptr(), b, s, heads, kshape[2], hd,
            *strides, *so, _dt(q), st))
    return o, lse


def masked_attention_backward(q, k, v, key_range, o, lse, do, scale: float | None = None, softcap: float = 0.0,
                              slopes=None, dq=None, dk=None, dv=None, stream=None):
    """Runs tpmlp_masked_attention_backward from do = dl/do (o's strides); allocates the workspace and, unless given,
    dq, dk and dv. Returns (dq, dk, dv)."""
    shape, kshape, strides = _masked_args(q, k, v, key_range, slopes)
    b, s, heads, hd = shape
    dtype = q.dtype
    _dense(lse, (b, heads, s), torch.float32, "lse")
    so = _heads(o, shape, dtype, "o")
    if _heads(do, shape, dtype, "do") != so:
        raise ValueError("do must have o's strides")
    lib = load_library()
    here, st = _where(_device(q, k, v, key_range, slopes, o, lse, do, dq, dk, dv), stream)
    with here:
        dq, sq = _out(dq, shape, q, "dq")
        dk, sk = _out(dk, kshape, q, "dk")
        dv, sv = _out(dv, kshape, q, "dv")
        ws_bytes = lib.tpmlp_masked_attention_backward_workspace_size(b, s, heads)
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
        _check(lib.tpmlp_masked_attention_backward(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), key_range.data_ptr(), _ptr(slopes),
            hd ** -0.5 if scale is None else scale, softcap, o.data_ptr(), lse.data_ptr(), do.data_ptr(), dq.data_ptr(),
            dk.data_ptr(), dv.data_ptr(), b, s, heads, kshape[2], hd, *strides, *so, *sq, *sk, *sv, _dt(q), ws.data_ptr(),
            ws_bytes, st))
    return dq, dk, dv


# ----------------------------------------------------------------------- gated feed-forward block

def _matrix(t: torch.Tensor, rows: int, cols: int, dtype: torch.dtype, name: str) -> None:
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or shape[1] != cols or t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {[rows, cols]}")


def _gated_args(X, A, B):
    n, d = X.shape
    m = B.shape[0]
    dtype = X.dtype
    _matrix(X, n, d, dtype, "X")
    _matrix(A, d, 2 * m, dtype, "A")
    _matrix(B, m, d, dtype, "B")
    return n, d, m, _dt(X)


def _scratch(nbytes: int, like: torch.Tensor):
    """A workspace of nbytes on like's device and its address; none for 0 bytes."""
    if nbytes == 0:
        return None, None
    ws = torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    return ws, ws.data_ptr()


def gated_forward(X, A, B, t: int = 1, act: str = "silu", save: bool = True, stream=None):
    """X [n, d], A [d, 2m] (shard by shard [gate | up]), B [m, d], bf16. Allocates O, Y and, with `save`, Z and runs
    tpmlp_gated_forward. Returns (O, Z or None, Y); gated_backward needs Z and Y."""
    n, d, m, dt = _gated_args(X, A, B)
    lib = load_library()
    here, st = _where(_device(X, A, B), stream)
    with here:
        O = torch.empty_like(X)
        Z = torch.empty((n, 2 * m), dtype=X.dtype, device=X.device) if save else None
        Y = torch.empty((n, m), dtype=X.dtype, device=X.device)
        ws_bytes = lib.tpmlp_gated_forward_workspace_size(n, d, m, t, dt)
        ws, ws_ptr = _scratch(ws_bytes, X)
        _check(lib.tpmlp_gated_forward(X.data_ptr(), A.data_ptr(), B.data_ptr(), O.data_ptr(), _ptr(Z), Y.data_ptr(), n, d,
                                       m, t, GATE_ACT[act], dt, ws_ptr, ws_bytes, st))
    return O, Z, Y


def gated_backward(X, A, B, G, Z, Y, t: int = 1, act: str = "silu", wgrad: str = "f32", dA=None, dB=None, stream=None):
    """Runs tpmlp_gated_backward from G = dl/dO and the forward's Z and Y; allocates dX, the workspace and, unless given,
    dA and dB. wgrad: "f32" (overwritten), "f32_add" (added to the given dA and dB) or "operand" (bf16). Returns
    (dX, dA, dB)."""
    n, d, m, dt = _gated_args(X, A, B)
    dtype = X.dtype
    _matrix(G, n, d, dtype, "G")
    _matrix(Z, n, 2 * m, dtype, "Z")
    _matrix(Y, n, m, dtype, "Y")
    act_kind, mode = GATE_ACT[act], WGRAD[wgrad]
    wtype = dtype if wgrad == "operand" else torch.float32
    if wgrad == "f32_add" and (dA is None or dB is None):
        raise ValueError("f32_add needs dA and dB")
    if dA is not None:
        _matrix(dA, d, 2 * m, wtype, "dA")
    if dB is not None:
        _matrix(dB, m, d, wtype, "dB")
    lib = load_library()
    here, st = _where(_device(X, A, B, G, Z, Y, dA, dB), stream)
    with here:
        dX = torch.empty_like(X)
        dA = torch.empty_like(A, dtype=wtype) if dA is None else dA
        dB = torch.empty_like(B, dtype=wtype) if dB is None else dB
        ws_bytes = lib.tpmlp_gated_backward_workspace_size(n, d, m, dt)
        ws, ws_ptr = _scratch(ws_bytes, X)
        _check(lib.tpmlp_gated_backward(X.data_ptr(), A.data_ptr(), B.data_ptr(), G.data_ptr(), Z.data_ptr(), Y.data_ptr(),
                                        dX.data_ptr(), dA.data_ptr(), dB.data_ptr(), n, d, m, t, act_kind, mode, dt,
                                        ws_ptr, ws_bytes, st))
    return dX, dA, dB


# ----------------------------------------------------------------------- norms around a block

def _gain(g: torch.Tensor, h: int, name: str) -> None:
    if g.dim() != 1 or g.numel() != h or g.dtype is not torch.float32 or not g.is_contiguous():
        raise ValueError(f"{name} must be a contiguous torch.float32 tensor of shape {[h]}")


def _residual_args(y, gamma_post, gate, gamma_pre):
    """(b, s, h) that the gate's rows divide the tokens of y [..., h] into."""
    shape = y.shape
    h = shape[-1]
    if gamma_post is not None:
        _gain(gamma_post, h, "gamma_post")
    if gamma_pre is not None:
        _gain(gamma_pre, h, "gamma_pre")
    tokens = y.numel() // h if h else 0
    if gate is None:
        return 1, tokens, h
    if gate.dim() == 1:
        _gain(gate, h, "gate")
        return 1, tokens, h
    if len(shape) < 3:
        raise ValueError("a gate of [b, h] needs tensors of [b, ..., h]")
    b = shape[0]
    _matrix(gate, b, h, torch.float32, "gate")
    return b, tokens // b if b else 0, h


def _alike(t: torch.Tensor, shape: torch.Size, dtype: torch.dtype, name: str) -> None:
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)}")


def residual_norm(x, y, gamma_post=None, gate=None, gamma_pre=None, alpha: float = 1.0, eps: float = 1e-5, r=None, u=None,
                  stream=None):
    """x (the residual) and y (a block's output) [..., h]; gains fp32 [h]; gate fp32 [h], or [b, h] for tensors [b, ..., h].
    Allocates r and u unless given (x or y for in place) and runs tpmlp_residual_norm. Returns (r, u), u None without
    gamma_pre."""
    shape, dtype = y.shape, y.dtype
    _alike(y, shape, dtype, "y")
    _alike(x, shape, dtype, "x")
    if r is not None:
        _alike(r, shape, dtype, "r")
    if u is not None:
        _alike(u, shape, dtype, "u")
        if gamma_pre is None:
            raise ValueError("u needs gamma_pre")
    b, s, h = _residual_args(y, gamma_post, gate, gamma_pre)
    dt = _dt(y)
    lib = load_library()
    here, st = _where(_device(y, x, gamma_post, gate, gamma_pre, r, u), stream)
    with here:
        r = torch.empty_like(y) if r is None else r
        u = torch.empty_like(y) if u is None and gamma_pre is not None else u
        _check(lib.tpmlp_residual_norm(x.data_ptr(), y.data_ptr(), _ptr(gamma_post), _ptr(gate), _ptr(gamma_pre), alpha, eps,
                                       r.data_ptr(), _ptr(u), b, s, h, dt, st))
    return r, u


def residual_norm_backward(y, r, dr, du, gamma_post=None, gate=None, gamma_pre=None, alpha: float = 1.0, eps: float = 1e-5,
                           dx=None, dy=None, stream=None):
    """Runs tpmlp_residual_norm_backward from dr = dl/dr and du = dl/du (either may be None: du without gamma_pre, dr beside
    du); r may be None without gamma_pre. Allocates the workspace, the gains' and the gate's gradients and, unless given,
    dx and dy. Returns (dx, dy, dgamma_post, dgate, dgamma_pre), None for a gain or gate that is not there."""
    like = y if y is not None else dr if dr is not None else du
    shape, dtype = like.shape, like.dtype
    for t, name in ((y, "y"), (r, "r"), (dr, "dr"), (du, "du"), (dx, "dx"), (dy, "dy")):
        if t is not None and (t.shape != shape or t.dtype is not dtype or not t.is_contiguous()):
            _alike(t, shape, dtype, name)
    b, s, h = _residual_args(like, gamma_post, gate, gamma_pre)
    dt = _dt(like)
    lib = load_library()
    here, st = _where(_device(like, r, dr, du, gamma_post, gate, gamma_pre, dx, dy), stream)
    with here:
        dx = torch.empty_like(like) if dx is None else dx
        dy = torch.empty_like(like) if dy is None else dy
        dpost = None if gamma_post is None else torch.empty_like(gamma_post)
        dgate = None if gate is None else torch.empty_like(gate)
        dpre = None if gamma_pre is None else torch.empty_like(gamma_pre)
        ws_bytes = lib.tpmlp_residual_norm_backward_workspace_size(b, s, h, gate is not None)
        ws, ws_ptr = _scratch(ws_bytes, like)
        _check(lib.tpmlp_residual_norm_backward(_ptr(y), _ptr(r), _ptr(dr), _ptr(du), _ptr(gamma_post), _ptr(gate),
                                                _ptr(gamma_pre), alpha, eps, dx.data_ptr(), dy.data_ptr(), _ptr(dpost),
                                                _ptr(dgate), _ptr(dpre), b, s, h, dt, ws_ptr, ws_bytes, st))
    return dx, dy, dpost, dgate, dpre
