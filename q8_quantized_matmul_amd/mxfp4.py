"""Python binding of include/mxfp4.h: the MXFP4 operators and the MoE router.

As in the package's other calls, torch supplies device memory and streams, and
all computation happens behind the C ABI.  A call runs on the device that
holds its tensors, on torch's current stream of that device; outputs and
scratch are allocated with torch when the caller passes none.  Everything here
is also available from the package itself.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import Q8Error, _i32, _i64, _lib, _sz, _vp

MXFP4_BLOCK_ELEMS = 32
MXFP4_F32, MXFP4_BF16, MXFP4_F16 = 0, 1, 2
MOE_SOFTMAX, MOE_SIGMOID, MOE_SQRT_SOFTPLUS = 0, 1, 2
_TYPES = {torch.float32: MXFP4_F32, torch.bfloat16: MXFP4_BF16, torch.float16: MXFP4_F16}

_sig = {
    "mxfp4_quantize": ([_vp, _vp, _vp, _i32, _i64, _i64, _i64, _vp], ctypes.c_int),
    "mxfp4_dequantize": ([_vp, _i32, _vp, _vp, _i64, _i64, _vp], ctypes.c_int),
    "moe_topk": ([_vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i32, ctypes.c_float, _vp],
                 ctypes.c_int),
}
for _name, (_args, _res) in _sig.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res

EXPORTED = tuple(_sig)


class Mxfp4(NamedTuple):
    """An MXFP4 matrix [..., k]: codes uint8 [..., k/2] (two values a byte, the
    even one in the low half) and e8m0 scale bytes uint8 [..., k/32]."""
    codes: torch.Tensor
    scales: torch.Tensor


def _type(dtype, name: str) -> int:
    t = _TYPES.get(dtype)
    if t is None:
        raise ValueError(f"{name} must be float32, bfloat16 or float16")
    return t


def _ptr(t: torch.Tensor, name: str, dtype, device) -> int:
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _device(t: torch.Tensor, name: str) -> torch.device:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.device


def _shape(t: torch.Tensor, name: str, *shape) -> None:
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")


def _matrix(m, name: str, device):
    """(codes pointer, scales pointer, leading shape, k) of an MXFP4 matrix."""
    codes, scales = m
    k = 2 * codes.shape[-1]
    if k % MXFP4_BLOCK_ELEMS != 0 or scales.shape != codes.shape[:-1] + (k // MXFP4_BLOCK_ELEMS,):
        raise ValueError(f"{name}: codes {list(codes.shape)} and scales {list(scales.shape)} are "
                         "not the two arrays of one matrix ([..., k/2] and [..., k/32])")
    return (_ptr(codes, name + ".codes", torch.uint8, device),
            _ptr(scales, name + ".scales", torch.uint8, device), codes.shape[:-1], k)


def _run(where: str, device, *args) -> None:
    """The C call with torch's current stream of `device` as its last argument."""
    index = device.index
    if index == torch.cuda.current_device():
        code = getattr(_lib, where)(*args, torch.cuda.current_stream(index).cuda_stream)
    else:
        with torch.cuda.device(index):
            code = getattr(_lib, where)(*args, torch.cuda.current_stream(index).cuda_stream)
    if code != 0:
        raise Q8Error(code, where)


def mxfp4_quantize(x: torch.Tensor, codes: torch.Tensor = None,
                   scales: torch.Tensor = None) -> Mxfp4:
    """MXFP4 rows of x (float32, bfloat16 or float16 [rows][k] or [k], k a
    multiple of 32; rows may lie any stride >= k apart)."""
    if x.dim() == 1:
        x = x.unsqueeze(0)
    if x.dim() != 2:
        raise ValueError("x must be [rows][k]")
    device = _device(x, "x")
    rows, k = x.shape
    stride = x.stride(0) if rows > 1 else k
    if k > 1 and x.stride(1) != 1:
        raise ValueError("the values of a row of x must be adjacent")
    if k % MXFP4_BLOCK_ELEMS != 0:
        raise ValueError("k must be a multiple of 32")
    if codes is None:
        codes = torch.empty((rows, k // 2), dtype=torch.uint8, device=device)
    if scales is None:
        scales = torch.empty((rows, k // MXFP4_BLOCK_ELEMS), dtype=torch.uint8, device=device)
    c, s, lead, k_out = _matrix((codes, scales), "out", device)
    if lead.numel() != rows or k_out != k:
        raise ValueError("codes and scales must hold as many rows and values as x")
    _run("mxfp4_quantize", device, c, s, x.data_ptr(), _type(x.dtype, "x"), stride, rows, k)
    return Mxfp4(codes, scales)


def mxfp4_dequantize(m: Mxfp4, dtype: torch.dtype = torch.float32,
                     out: torch.Tensor = None) -> torch.Tensor:
    """The values [..., k] that an MXFP4 matrix stands for (exact in float32 and bfloat16)."""
    device = _device(m[0], "codes")
    c, s, lead, k = _matrix(m, "m", device)
    if out is None:
        out = torch.empty((*lead, k), dtype=dtype, device=device)
    _shape(out, "out", *lead, k)
    _run("mxfp4_dequantize", device, _ptr(out, "out", out.dtype, device), _type(out.dtype, "out"),
         c, s, lead.numel(), k)
    return out


def moe_topk(logits: torch.Tensor, n_used: int, bias: torch.Tensor = None,
             scoring: int = MOE_SOFTMAX, renormalize: bool = True, scale: float = 1.0,
             selected: torch.Tensor = None, weights: torch.Tensor = None):
    """(selected int32, weights float32), both [n_tok][n_used]: each token's experts of
    largest score + bias from float32 logits [n_tok][n_expert].  Slots without an
    eligible expert (logits of -inf) hold id -1 and weight 0."""
    if logits.dim() != 2:
        raise ValueError("logits must be [n_tok][n_expert]")
    device = _device(logits, "logits")
    n_tok, n_expert = logits.shape
    if selected is None:
        selected = torch.empty((n_tok, n_used), dtype=torch.int32, device=device)
    if weights is None:
        weights = torch.empty((n_tok, n_used), dtype=torch.float32, device=device)
    _shape(selected, "selected", n_tok, n_used)
    _shape(weights, "weights", n_tok, n_used)
    if bias is not None:
        _shape(bias, "bias", n_expert)
        bias = _ptr(bias, "bias", torch.float32, device)
    _run("moe_topk", device, _ptr(selected, "selected", torch.int32, device),
         _ptr(weights, "weights", torch.float32, device),
         _ptr(logits, "logits", torch.float32, device), bias, n_tok, n_expert, n_used, scoring,
         int(renormalize), scale)
    return selected, weights
