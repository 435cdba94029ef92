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
_I32_MAX = 2 ** 31 - 1
_TYPES = {torch.float32: MXFP4_F32, torch.bfloat16: MXFP4_BF16, torch.float16: MXFP4_F16}

class MoeLayerArgs(ctypes.Structure):
    """struct mxfp4_moe_layer_args."""
    _fields_ = [("out", _vp), ("x", _vp), ("out_type", _i32), ("x_type", _i32), ("logits", _vp),
                ("bias", _vp), ("n_expert", _i32), ("n_used", _i32), ("scoring", _i32),
                ("renormalize", _i32), ("scale", ctypes.c_float), ("clamp", ctypes.c_float),
                ("d_model", _i64), ("d_ff", _i64), ("n_tok", _i64), ("gate_codes", _vp),
                ("gate_scales", _vp), ("up_codes", _vp), ("up_scales", _vp), ("down_codes", _vp),
                ("down_scales", _vp), ("selected", _vp), ("weights", _vp)]


_sig = {
    "mxfp4_quantize": ([_vp, _vp, _vp, _i32, _i64, _i64, _i64, _vp], ctypes.c_int),
    "mxfp4_dequantize": ([_vp, _i32, _vp, _vp, _i64, _i64, _vp], ctypes.c_int),
    "mxfp4_matmul_workspace_bytes": ([_i64, _i64, _i64], _sz),
    "mxfp4_matmul": ([_vp, _i32, _vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _sz, _vp],
                     ctypes.c_int),
    "moe_topk": ([_vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i32, ctypes.c_float, _vp],
                 ctypes.c_int),
    "mxfp4_moe_layer_workspace_bytes": ([_i64, _i32, _i32, _i64, _i64], _sz),
    "mxfp4_moe_layer": ([ctypes.POINTER(MoeLayerArgs), _vp, _sz, _vp], ctypes.c_int),
}
for _name, (_args, _res) in _sig.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res

EXPORTED = tuple(_sig)
_calls = {_name: getattr(_lib, _name) for _name in EXPORTED}


class Mxfp4(NamedTuple):
    """An MXFP4 matrix [..., k]: codes uint8 [..., k/2] (two values a byte, the
    even one in the low half) and e8m0 scale bytes uint8 [..., k/32]."""
    codes: torch.Tensor
    scales: torch.Tensor


# A decode step makes these calls by the hundred: the raw forms of torch.cuda's
# current device and stream cost a tenth of the public ones, and torch.empty takes
# its sizes in 1.3 us one by one and in 1.7 as a tuple.
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


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
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")


def _route_sizes(n_expert: int, n_used: int, scoring: int) -> None:
    """Refuses what the C call's 32-bit arguments would take for another number."""
    if n_expert > _I32_MAX or n_used > _I32_MAX or scoring > _I32_MAX:
        raise ValueError("n_expert, n_used and scoring must be below 2^31")


def _matrix(m, name: str, device):
    """(codes pointer, scales pointer, leading shape, k) of an MXFP4 matrix."""
    codes, scales = m
    cs, ss = codes.shape, scales.shape
    lead = cs[:-1]
    if not cs or not ss or cs[-1] != 16 * ss[-1] or lead != ss[:-1]:
        raise ValueError(f"{name}: codes {list(cs)} and scales {list(ss)} are not the two arrays of "
                         "one matrix ([..., k/2] and [..., k/32])")
    if not (codes.dtype == scales.dtype == torch.uint8 and codes.device == scales.device == device
            and codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError(f"{name}: codes and scales must be contiguous uint8 on {device}")
    return codes.data_ptr(), scales.data_ptr(), lead, 2 * cs[-1]


def _run(where: str, device, *args) -> None:
    """The C call with torch's current stream of `device` as its last argument."""
    index = device.index
    if index == _current_device():
        code = _calls[where](*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            code = _calls[where](*args, _raw_stream(index))
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
    stride, one = x.stride()
    if rows <= 1:
        stride = k
    if one != 1 and k > 1:
        raise ValueError("the values of a row of x must be adjacent")
    if k % MXFP4_BLOCK_ELEMS != 0:
        raise ValueError("k must be a multiple of 32")
    given = codes is not None or scales is not None
    if codes is None:
        codes = torch.empty(rows, k // 2, dtype=torch.uint8, device=device)
    if scales is None:
        scales = torch.empty(rows, k // MXFP4_BLOCK_ELEMS, dtype=torch.uint8, device=device)
    out = Mxfp4(codes, scales)
    if given:
        _, _, lead, k_out = _matrix(out, "out", device)
        if k_out != k or lead.numel() != rows:
            raise ValueError("codes and scales must hold as many rows and values as x")
    c, s = codes.data_ptr(), scales.data_ptr()
    _run("mxfp4_quantize", device, c, s, x.data_ptr(), _type(x.dtype, "x"), stride, rows, k)
    return out


def mxfp4_dequantize(m: Mxfp4, dtype: torch.dtype = torch.float32,
                     out: torch.Tensor = None) -> torch.Tensor:
    """The values [..., k] that an MXFP4 matrix stands for: exact in float32 and bfloat16
    but for values of 2^128 and above (scale bytes 253 and 254), which are infinite."""
    device = _device(m[0], "codes")
    c, s, lead, k = _matrix(m, "m", device)
    if out is None:
        out = torch.empty(*lead, k, dtype=dtype, device=device)
        o = out.data_ptr()
    else:
        _shape(out, "out", *lead, k)
        dtype = out.dtype
        o = _ptr(out, "out", dtype, device)
    _run("mxfp4_dequantize", device, o, _type(dtype, "out"), c, s, lead.numel(), k)
    return out


def mxfp4_matmul_workspace_bytes(in_dim: int, out_dim: int, n_tok: int) -> int:
    return int(_lib.mxfp4_matmul_workspace_bytes(in_dim, out_dim, n_tok))


def mxfp4_matmul_workspace(in_dim: int, out_dim: int, n_tok: int, device="cuda") -> torch.Tensor:
    """Scratch for mxfp4_matmul calls of this shape (contents do not matter)."""
    return torch.empty(mxfp4_matmul_workspace_bytes(in_dim, out_dim, n_tok), dtype=torch.uint8,
                       device=device)


def _scratch(t, need: int, device):
    """(pointer, bytes) of the caller's scratch, or of `need` bytes allocated now; the
    allocator keeps a freed tensor's memory for later work on the same stream."""
    if t is None:
        if need == 0:
            return None, 0, None
        t = torch.empty(need, dtype=torch.uint8, device=device)
        return t.data_ptr(), need, t
    return _ptr(t, "workspace", torch.uint8, device), t.numel(), t


def mxfp4_matmul(w: Mxfp4, x: Mxfp4, out: torch.Tensor = None,
                 out_dtype: torch.dtype = torch.float32,
                 workspace: torch.Tensor = None) -> torch.Tensor:
    """out [n_tok][out_dim] = x [n_tok][k] times w [out_dim][k] transposed, both MXFP4,
    as float32 (or out_dtype, or out's type).  Without a workspace one is
    allocated for shapes that can use it."""
    device = _device(x[0], "x.codes")
    wc, wsc, w_lead, k = _matrix(w, "w", device)
    xc, xsc, x_lead, xk = _matrix(x, "x", device)
    if len(w_lead) != 1 or len(x_lead) != 1 or xk != k:
        raise ValueError("w must be [out_dim][k] and x [n_tok][k]")
    out_dim, n_tok = w_lead[0], x_lead[0]
    if out is None:
        out = torch.empty(n_tok, out_dim, dtype=out_dtype, device=device)
        o = out.data_ptr()
    else:
        _shape(out, "out", n_tok, out_dim)
        out_dtype = out.dtype
        o = _ptr(out, "out", out_dtype, device)
    ws, ws_bytes, keep = _scratch(workspace, mxfp4_matmul_workspace_bytes(k, out_dim, n_tok)
                                  if workspace is None else 0, device)
    _run("mxfp4_matmul", device, o, _type(out_dtype, "out"), wc, wsc, k, out_dim, xc, xsc, n_tok, ws,
         ws_bytes)
    return out


def _routing(selected, weights, n_tok: int, n_used: int, device):
    """(selected, its pointer, weights, its pointer), allocated where not given."""
    if selected is None:
        selected = torch.empty(n_tok, n_used, dtype=torch.int32, device=device)
        sp = selected.data_ptr()
    else:
        _shape(selected, "selected", n_tok, n_used)
        sp = _ptr(selected, "selected", torch.int32, device)
    if weights is None:
        weights = torch.empty(n_tok, n_used, dtype=torch.float32, device=device)
        wp = weights.data_ptr()
    else:
        _shape(weights, "weights", n_tok, n_used)
        wp = _ptr(weights, "weights", torch.float32, device)
    return selected, sp, weights, wp


def moe_topk(logits: torch.Tensor, n_used: int, bias: torch.Tensor = None,
             scoring: int = MOE_SOFTMAX, renormalize: bool = True, scale: float = 1.0,
             selected: torch.Tensor = None, weights: torch.Tensor = None):
    """(selected int32, weights float32), both [n_tok][n_used]: each token's experts of
    largest score + bias from float32 logits [n_tok][n_expert]; for MOE_SOFTMAX of
    largest logit + bias, which a bias on the probabilities does not equal.  Slots
    without an eligible expert (logits of -inf) hold id -1 and weight 0."""
    if logits.dim() != 2:
        raise ValueError("logits must be [n_tok][n_expert]")
    device = _device(logits, "logits")
    n_tok, n_expert = logits.shape
    _route_sizes(n_expert, n_used, scoring)
    selected, sp, weights, wp = _routing(selected, weights, n_tok, n_used, device)
    if bias is not None:
        _shape(bias, "bias", n_expert)
        bias = _ptr(bias, "bias", torch.float32, device)
    _run("moe_topk", device, sp, wp, _ptr(logits, "logits", torch.float32, device), bias, n_tok,
         n_expert, n_used, scoring, int(renormalize), scale)
    return selected, weights


def mxfp4_moe_layer_workspace_bytes(n_tok: int, n_used: int, n_expert: int, d_model: int,
                                    d_ff: int) -> int:
    _route_sizes(n_expert, n_used, 0)
    return int(_lib.mxfp4_moe_layer_workspace_bytes(n_tok, n_used, n_expert, d_model, d_ff))


def mxfp4_moe_layer_workspace(n_tok: int, n_used: int, n_expert: int, d_model: int, d_ff: int,
                              device="cuda") -> torch.Tensor:
    """Scratch for mxfp4_moe_layer calls of these sizes (contents do not matter)."""
    n = mxfp4_moe_layer_workspace_bytes(n_tok, n_used, n_expert, d_model, d_ff)
    return torch.empty(n, dtype=torch.uint8, device=device)


def mxfp4_moe_layer(x: torch.Tensor, logits: torch.Tensor, gate: Mxfp4, up: Mxfp4, down: Mxfp4,
                    n_used: int, bias: torch.Tensor = None, scoring: int = MOE_SOFTMAX,
                    renormalize: bool = True, scale: float = 1.0, clamp: float = 0.0,
                    out: torch.Tensor = None, out_dtype: torch.dtype = None,
                    selected: torch.Tensor = None, weights: torch.Tensor = None,
                    workspace: torch.Tensor = None):
    """The whole MoE layer for up to 64 tokens: x (float32, bfloat16 or float16
    [n_tok][d_model]) and router logits (float32 [n_tok][n_expert]) through the
    chosen experts' MXFP4 matrices gate, up [n_expert][d_ff][d_model] and down
    [n_expert][d_model][d_ff].  Returns (out [n_tok][d_model] of out_dtype, by
    default x's, selected, weights), the last two as moe_topk gives them."""
    device = _device(x, "x")
    if x.dim() != 2 or logits.dim() != 2:
        raise ValueError("x must be [n_tok][d_model] and logits [n_tok][n_expert]")
    n_tok, d_model = x.shape
    n_expert = logits.shape[1]
    _route_sizes(n_expert, n_used, scoring)
    gc, gs, g_lead, gk = _matrix(gate, "gate", device)
    uc, us, u_lead, uk = _matrix(up, "up", device)
    dc, ds, d_lead, d_ff = _matrix(down, "down", device)
    if (tuple(g_lead) != (n_expert, d_ff) or tuple(u_lead) != (n_expert, d_ff)
            or tuple(d_lead) != (n_expert, d_model) or gk != d_model or uk != d_model
            or logits.shape[0] != n_tok):
        raise ValueError("x [n_tok][d_model], logits [n_tok][n_expert], gate and up [n_expert][d_ff]"
                         "[d_model] and down [n_expert][d_model][d_ff] do not fit together")
    if bias is not None:
        _shape(bias, "bias", n_expert)
        bias = _ptr(bias, "bias", torch.float32, device)
    if out is None:
        out = torch.empty(n_tok, d_model, dtype=out_dtype or x.dtype, device=device)
    else:
        _shape(out, "out", n_tok, d_model)
    selected, sp, weights, wp = _routing(selected, weights, n_tok, n_used, device)
    ws, ws_bytes, keep = _scratch(
        workspace, mxfp4_moe_layer_workspace_bytes(n_tok, n_used, n_expert, d_model, d_ff)
        if workspace is None else 0, device)
    args = MoeLayerArgs(_ptr(out, "out", out.dtype, device), _ptr(x, "x", x.dtype, device),
                        _type(out.dtype, "out"), _type(x.dtype, "x"),
                        _ptr(logits, "logits", torch.float32, device), bias, n_expert, n_used,
                        scoring, int(renormalize), scale, clamp, d_model, d_ff, n_tok, gc, gs, uc,
                        us, dc, ds, sp, wp)
    _run("mxfp4_moe_layer", device, ctypes.byref(args), ws, ws_bytes)
    return out, selected, weights
