"""Python binding of include/kv8.h: the 8-bit key/value cache and attention over it.

As in the package's other calls, torch supplies device memory and streams, and
all computation happens behind the C ABI.  A Kv8Cache holds one layer's pool of
pages, a Kv8Batch one step's sequences; both look their tensors over once, so
that the calls of a step's layers, which share the batch, need not.  A call runs
on the device that holds its tensors, on torch's current stream of that device.
Everything here is also available from the package itself.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _i32, _i64, _lib, _sz, _vp
from .mxfp4 import _calls, _device, _ptr, _run, _scratch, _shape, _type

KV8_F32, KV8_BF16, KV8_F16 = 0, 1, 2
KV8_KERNEL_AUTO, KV8_KERNEL_STREAM, KV8_KERNEL_TILED = 0, 1, 2
_I32_MAX = 2 ** 31 - 1


class _CacheArgs(ctypes.Structure):
    """struct kv8_cache."""
    _fields_ = [("k_codes", _vp), ("v_codes", _vp), ("k_scales", _vp), ("v_scales", _vp),
                ("n_pages", _i64), ("n_kv", _i32), ("head_dim", _i32), ("page_size", _i32),
                ("block", _i32)]


class _BatchArgs(ctypes.Structure):
    """struct kv8_batch."""
    _fields_ = [("page_table", _vp), ("lens", _vp), ("starts", _vp), ("n_seq", _i64),
                ("n_tok", _i64), ("table_width", _i64), ("max_new", _i64), ("max_len", _i64)]


class _AttentionArgs(ctypes.Structure):
    """struct kv8_attention_args."""
    _fields_ = [("out", _vp), ("q", _vp), ("q_token_stride", _i64), ("q_head_stride", _i64),
                ("out_type", _i32), ("q_type", _i32), ("n_q", _i32), ("window", _i32),
                ("scale", ctypes.c_float), ("sinks", _vp), ("lse", _vp)]


_sig = {
    "kv8_write": ([_vp, _vp, _vp, _i64, _i64, _vp, _i64, _i64, _i32, _vp], ctypes.c_int),
    "kv8_read": ([_vp, _vp, _vp, _vp, _i32, _vp], ctypes.c_int),
    "kv8_attention_workspace_bytes": ([_vp, _vp, _i32], _sz),
    "kv8_attention": ([_vp, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    "kv8_attention_debug": ([_vp, _vp, _vp, _vp, _sz, _i32, _i32, _vp], ctypes.c_int),
}
for _name, (_args, _res) in _sig.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res
    _calls[_name] = _fn

EXPORTED = tuple(_sig)


class Kv8Cache:
    """A pool of pages: int8 codes k, v [n_pages][n_kv][page_size][head_dim] (in the order that
    kv8.h gives, not token by token) and float32 scales k_scales, v_scales
    [n_pages][n_kv][page_size / block]."""
    __slots__ = ("k", "v", "k_scales", "v_scales", "n_pages", "n_kv", "head_dim", "page_size",
                 "block", "device", "_args", "_ref")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scales: torch.Tensor,
                 v_scales: torch.Tensor):
        self.device = _device(k, "k")
        if k.dim() != 4 or k_scales.dim() != 3 or 0 in k_scales.shape:
            raise ValueError("codes must be [n_pages][n_kv][page_size][head_dim] and scales "
                             "[n_pages][n_kv][page_size / block]")
        self.n_pages, self.n_kv, self.page_size, self.head_dim = k.shape
        blocks = k_scales.shape[2]
        if self.page_size % blocks != 0:
            raise ValueError("the page size must be a multiple of the scales of a page")
        self.block = self.page_size // blocks
        _shape(v, "v", *k.shape)
        for t, name in ((k_scales, "k_scales"), (v_scales, "v_scales")):
            _shape(t, name, self.n_pages, self.n_kv, blocks)
        if max(k.shape) > _I32_MAX:
            raise ValueError("sizes of a cache must be below 2^31")
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self._args = _CacheArgs(_ptr(k, "k", torch.int8, self.device),
                                _ptr(v, "v", torch.int8, self.device),
                                _ptr(k_scales, "k_scales", torch.float32, self.device),
                                _ptr(v_scales, "v_scales", torch.float32, self.device),
                                self.n_pages, self.n_kv, self.head_dim, self.page_size, self.block)
        self._ref = ctypes.addressof(self._args)


def kv8_cache(n_pages: int, n_kv: int, head_dim: int, page_size: int = 64, block: int = 16,
              device="cuda") -> Kv8Cache:
    """An empty cache (zero codes and scales)."""
    if block < 1 or page_size % block != 0:
        raise ValueError("page_size must be a multiple of block")
    codes = (torch.zeros(n_pages, n_kv, page_size, head_dim, dtype=torch.int8, device=device)
             for _ in range(2))
    scales = (torch.zeros(n_pages, n_kv, page_size // block, device=device) for _ in range(2))
    return Kv8Cache(*codes, *scales)


class Kv8Batch:
    """A step's sequences: int32 page_table [n_seq][pages], lens [n_seq] (tokens of each, the new
    ones among them) and starts [n_seq + 1], by which sequence s owns rows starts[s] ..
    starts[s + 1] - 1 of the step's n_tok rows, its newest tokens; without starts each
    sequence owns one row.  max_new: no sequence owns more rows (by default n_tok); max_len: no
    length is above it (by default the table's room).  The tensors are read when the calls
    run, so a captured step can be replayed with other contents."""
    __slots__ = ("page_table", "lens", "starts", "n_seq", "n_tok", "max_new", "max_len", "device",
                 "_args", "_ref")

    def __init__(self, page_table: torch.Tensor, lens: torch.Tensor, starts: torch.Tensor = None,
                 n_tok: int = None, max_new: int = None, max_len: int = None):
        self.device = _device(page_table, "page_table")
        if page_table.dim() != 2:
            raise ValueError("page_table must be [n_seq][pages]")
        self.n_seq, width = page_table.shape
        _shape(lens, "lens", self.n_seq)
        if starts is None:
            if n_tok not in (None, self.n_seq) or max_new not in (None, 1):
                raise ValueError("without starts every sequence owns one row")
            n_tok, max_new, sp = self.n_seq, 1, None
        else:
            if n_tok is None:
                raise ValueError("n_tok must be given with starts")
            _shape(starts, "starts", self.n_seq + 1)
            sp = _ptr(starts, "starts", torch.int32, self.device)
        self.n_tok = n_tok
        self.max_new = n_tok if max_new is None else max_new
        self.max_len = max_len or 0
        if min(self.n_tok, self.max_new, self.max_len) < 0:
            raise ValueError("n_tok, max_new and max_len must not be negative")
        if max(self.n_tok, self.max_new, self.max_len) > 2 ** 62:
            raise ValueError("n_tok, max_new and max_len must be below 2^62")
        self.page_table, self.lens, self.starts = page_table, lens, starts
        self._args = _BatchArgs(_ptr(page_table, "page_table", torch.int32, self.device),
                                _ptr(lens, "lens", torch.int32, self.device), sp, self.n_seq,
                                self.n_tok, width, self.max_new, self.max_len)
        self._ref = ctypes.addressof(self._args)


def _rows(t: torch.Tensor, name: str, n_tok: int, heads, d: int, device, dtype):
    """(pointer, token stride, head stride) of rows [n_tok][heads][d]."""
    shape = t.shape
    if len(shape) != 3 or shape[0] != n_tok or shape[2] != d or (heads and shape[1] != heads):
        raise ValueError(f"{name} must have shape [{n_tok}][{heads or 'heads'}][{d}], "
                         f"got {list(shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")
    token, head, one = t.stride()
    if one != 1:
        raise ValueError(f"the values of a head of {name} must be adjacent")
    return t.data_ptr(), token, head


def _same_device(cache: Kv8Cache, batch: Kv8Batch):
    if batch.device != cache.device:
        raise ValueError(f"the batch must be on {cache.device}")
    return cache.device


def kv8_write(cache: Kv8Cache, batch: Kv8Batch, k: torch.Tensor, v: torch.Tensor) -> None:
    """Write the batch's rows k, v (float32, bfloat16 or float16 [n_tok][n_kv][head_dim], any
    strides between tokens and between heads) into the cache: int8 under the scale of their block, older
    codes of the block rounded anew where its scale grows."""
    device = _same_device(cache, batch)
    dtype = k.dtype
    kp, kt, kh = _rows(k, "k", batch.n_tok, cache.n_kv, cache.head_dim, device, dtype)
    vp, vt, vh = _rows(v, "v", batch.n_tok, cache.n_kv, cache.head_dim, device, dtype)
    _run("kv8_write", device, cache._ref, batch._ref, kp, kt, kh, vp, vt, vh, _type(dtype, "k"))


def kv8_read(cache: Kv8Cache, batch: Kv8Batch, dtype: torch.dtype = torch.float32,
             k: torch.Tensor = None, v: torch.Tensor = None):
    """(k, v) [n_tok][n_kv][head_dim]: the values that the batch's rows have in the cache, as dtype
    or the type of the given outputs."""
    device = _same_device(cache, batch)
    shape = (batch.n_tok, cache.n_kv, cache.head_dim)
    if k is not None:
        dtype = k.dtype
        _shape(k, "k", *shape)
        kp = _ptr(k, "k", dtype, device)
    elif v is not None:
        dtype = v.dtype
    if k is None:
        k = torch.empty(*shape, dtype=dtype, device=device)
        kp = k.data_ptr()
    if v is None:
        v = torch.empty(*shape, dtype=dtype, device=device)
        vp = v.data_ptr()
    else:
        _shape(v, "v", *shape)
        vp = _ptr(v, "v", dtype, device)
    _run("kv8_read", device, cache._ref, batch._ref, kp, vp, _type(dtype, "out"))
    return k, v


def kv8_attention_workspace_bytes(cache: Kv8Cache, batch: Kv8Batch, n_q: int) -> int:
    if not 0 < n_q <= _I32_MAX:
        raise ValueError("n_q must be positive and below 2^31")
    return int(_lib.kv8_attention_workspace_bytes(cache._ref, batch._ref, n_q))


def kv8_attention_workspace(cache: Kv8Cache, batch: Kv8Batch, n_q: int) -> torch.Tensor:
    """Scratch for kv8_attention calls of these sizes (contents do not matter)."""
    return torch.empty(kv8_attention_workspace_bytes(cache, batch, n_q), dtype=torch.uint8,
                       device=cache.device)


def kv8_attention(cache: Kv8Cache, batch: Kv8Batch, q: torch.Tensor, scale: float = None,
                  window: int = 0, sinks: torch.Tensor = None, out: torch.Tensor = None,
                  out_dtype: torch.dtype = None, lse: torch.Tensor = None,
                  workspace: torch.Tensor = None) -> torch.Tensor:
    """out [n_tok][n_q][head_dim]: causal attention of the rows q (float32, bfloat16 or float16,
    any strides between tokens and between heads) over their sequences' cached tokens, their own
    among them, as q's type, out_dtype or out's type.  scale: by default 1 / sqrt(head_dim); window:
    keys that a row sees (0: all); sinks: float32 [n_q], a score per head that has no value;
    lse: float32 [n_tok][n_q], receives the log of each row's sum."""
    return _attend(cache, batch, q, scale, window, sinks, out, out_dtype, lse, workspace)


def kv8_attention_debug(cache: Kv8Cache, batch: Kv8Batch, q: torch.Tensor, kernel: int,
                        splits: int = 0, scale: float = None, window: int = 0,
                        sinks: torch.Tensor = None, out: torch.Tensor = None,
                        out_dtype: torch.dtype = None, lse: torch.Tensor = None,
                        workspace: torch.Tensor = None) -> torch.Tensor:
    """Test hook: kv8_attention by the given kernel (KV8_KERNEL_*) with that many splits."""
    if workspace is None:
        rows = batch.n_tok * (q.shape[1] if q.dim() > 1 else 0)
        need = splits * rows * (cache.head_dim + 1) * 4 if splits > 1 else 0
        workspace = torch.empty(need, dtype=torch.uint8, device=cache.device)
    return _attend(cache, batch, q, scale, window, sinks, out, out_dtype, lse, workspace,
                   "kv8_attention_debug", kernel, splits)


def _attend(cache, batch, q, scale, window, sinks, out, out_dtype, lse, workspace,
            call="kv8_attention", *choice):
    device = _same_device(cache, batch)
    d, n_tok, n_kv = cache.head_dim, batch.n_tok, cache.n_kv
    qp, qt, qh = _rows(q, "q", n_tok, 0, d, device, q.dtype)
    n_q = q.shape[1]
    if n_q < 1 or n_q % n_kv != 0:
        raise ValueError(f"the heads of q must be a multiple of {n_kv}")
    if not 0 <= window <= _I32_MAX or n_q > _I32_MAX:
        raise ValueError("window must be 0 .. 2^31 - 1")
    if out is None:
        out_dtype = out_dtype or q.dtype
        out = torch.empty(n_tok, n_q, d, dtype=out_dtype, device=device)
        op = out.data_ptr()
    else:
        _shape(out, "out", n_tok, n_q, d)
        out_dtype = out.dtype
        op = _ptr(out, "out", out_dtype, device)
    if sinks is not None:
        _shape(sinks, "sinks", n_q)
        sinks = _ptr(sinks, "sinks", torch.float32, device)
    if lse is not None:
        _shape(lse, "lse", n_tok, n_q)
        lse = _ptr(lse, "lse", torch.float32, device)
    ws, ws_bytes, keep = _scratch(workspace, kv8_attention_workspace_bytes(cache, batch, n_q)
                                  if workspace is None else 0, device)
    args = _AttentionArgs(op, qp, qt, qh, _type(out_dtype, "out"), _type(q.dtype, "q"), n_q, window,
                          1.0 / math.sqrt(d) if scale is None else scale, sinks, lse)
    _run(call, device, cache._ref, batch._ref, ctypes.byref(args), ws, ws_bytes, *choice)
    return out
