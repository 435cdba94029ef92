"""CPU checks of include/kv8.h: every declared function is exported and bound, and
the host-side argument checks refuse what the header says they refuse.  No call
here reaches a device: each fails validation, or is empty."""
import ctypes
import math
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # never dereferenced

CACHE = dict(k_codes=FAKE, v_codes=FAKE, k_scales=FAKE, v_scales=FAKE, n_pages=8, n_kv=2, head_dim=128, page_size=64,
             block=16)
BATCH = dict(page_table=FAKE, lens=FAKE, starts=FAKE, n_seq=2, n_tok=5, table_width=4, max_new=5, max_len=0)
BAD_CACHE = [dict(n_pages=0), dict(n_pages=-1), dict(n_pages=1 << 31), dict(n_kv=0), dict(n_kv=4097), dict(head_dim=96),
             dict(head_dim=0), dict(head_dim=1024), dict(page_size=8), dict(page_size=48), dict(page_size=2048),
             dict(block=8), dict(block=24), dict(block=128), dict(page_size=1024, block=256), dict(block=0)]
BAD_BATCH = [dict(n_seq=-1), dict(n_seq=(1 << 20) + 1), dict(n_tok=-1), dict(n_tok=(1 << 24) + 1), dict(table_width=-1),
             dict(table_width=(1 << 24) + 1), dict(max_new=-1), dict(max_len=-1), dict(starts=None)]
NULLS = [("cache", dict(k_codes=None)), ("cache", dict(v_codes=None)), ("cache", dict(k_scales=None)),
         ("cache", dict(v_scales=None)), ("batch", dict(lens=None)), ("batch", dict(page_table=None))]
MISALIGNED = [("cache", dict(k_codes=FAKE + 8)), ("cache", dict(v_codes=FAKE + 4)), ("cache", dict(k_scales=FAKE + 2)),
              ("cache", dict(v_scales=FAKE + 1)), ("batch", dict(lens=FAKE + 2)), ("batch", dict(page_table=FAKE + 2)),
              ("batch", dict(starts=FAKE + 2))]


@pytest.fixture(scope="module")
def q8():
    import q8_quantized_matmul_amd as m
    return m


@pytest.fixture(scope="module")
def calls(q8):
    from q8_quantized_matmul_amd import kv8
    lib = q8.raw_library()

    def structs(cache, batch):
        c, b = kv8._CacheArgs(**{**CACHE, **(cache or {})}), kv8._BatchArgs(**{**BATCH, **(batch or {})})
        return ctypes.byref(c), ctypes.byref(b), (c, b)

    def write(cache=None, batch=None, k=FAKE, kt=256, kh=128, v=FAKE, vt=256, vh=128, type=1):
        c, b, keep = structs(cache, batch)
        return lib.kv8_write(c, b, k, kt, kh, v, vt, vh, type, None)

    def read(cache=None, batch=None, k=FAKE, v=FAKE, type=1):
        c, b, keep = structs(cache, batch)
        return lib.kv8_read(c, b, k, v, type, None)

    def attention(cache=None, batch=None, ws=None, ws_bytes=0, **args):
        c, b, keep = structs(cache, batch)
        a = kv8._AttentionArgs(**{**dict(out=FAKE, q=FAKE, q_token_stride=1024, q_head_stride=128, out_type=1, q_type=1,
                                         n_q=8, window=0, scale=0.1, sinks=None, lse=None), **args})
        return lib.kv8_attention(c, b, ctypes.byref(a), ws, ws_bytes, None)

    def debug(cache=None, batch=None, ws=None, ws_bytes=0, kernel=1, splits=0, **args):
        c, b, keep = structs(cache, batch)
        a = kv8._AttentionArgs(**{**dict(out=FAKE, q=FAKE, q_token_stride=1024, q_head_stride=128, out_type=1, q_type=1,
                                         n_q=8, window=0, scale=0.1, sinks=None, lse=None), **args})
        return lib.kv8_attention_debug(c, b, ctypes.byref(a), ws, ws_bytes, kernel, splits, None)

    def workspace(cache=None, batch=None, n_q=8):
        c, b, keep = structs(cache, batch)
        return lib.kv8_attention_workspace_bytes(c, b, n_q)
    return dict(write=write, read=read, attention=attention, debug=debug, workspace=workspace)


def test_exports_every_declared_symbol(q8):
    from q8_quantized_matmul_amd import kv8
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "kv8.h")).read(), flags=re.S)
    declared = set(re.findall(r"\b(kv8_\w+)\s*\(", text))
    assert declared == set(kv8.EXPORTED)
    for name in declared:
        assert hasattr(ctypes.CDLL(q8.LIB_PATH), name) and hasattr(q8, name), name


@pytest.mark.parametrize("call", ["write", "read", "attention"])
def test_cache_and_batch_refusals(q8, calls, call):
    f = calls[call]
    for bad in BAD_CACHE:
        assert f(cache=bad) == q8.Q8_0_EINVAL, bad
    for bad in BAD_BATCH:
        assert f(batch=bad) == q8.Q8_0_EINVAL, bad
    assert f(cache=dict(n_kv=4096), batch=dict(n_seq=1025)) == q8.Q8_0_EINVAL
    for where, bad in NULLS:
        assert f(**{where: bad}) == q8.Q8_0_EINVAL, bad
    for where, bad in MISALIGNED:
        assert f(**{where: bad}) == q8.Q8_0_EALIGN, bad
    for empty in (dict(n_seq=0), dict(n_tok=0), dict(max_new=0), dict(n_seq=0, n_tok=0, starts=None)):
        assert f(batch=empty) == q8.Q8_0_OK, empty


def test_write_refusals(q8, calls):
    f = calls["write"]
    for bad in (dict(type=3), dict(type=-1), dict(kt=-1), dict(kh=-1), dict(vt=-1), dict(vh=-1), dict(k=None), dict(v=None),
                dict(kt=1 << 41)):
        assert f(**bad) == q8.Q8_0_EINVAL, bad
    for bad in (dict(k=FAKE + 1), dict(v=FAKE + 1), dict(k=FAKE + 2, type=0)):
        assert f(**bad) == q8.Q8_0_EALIGN, bad


def test_read_refusals(q8, calls):
    f = calls["read"]
    assert f(type=3) == q8.Q8_0_EINVAL
    assert f(k=FAKE + 8) == q8.Q8_0_EALIGN and f(v=FAKE + 2) == q8.Q8_0_EALIGN
    assert f(k=None, v=None) == q8.Q8_0_OK


def test_attention_refusals(q8, calls):
    f = calls["attention"]
    for bad in (dict(n_q=0), dict(n_q=7), dict(n_q=-2), dict(n_q=(1 << 14) + 2), dict(window=-1), dict(scale=math.inf),
                dict(scale=math.nan), dict(out_type=3), dict(q_type=-1), dict(q_token_stride=-1), dict(q_head_stride=-1),
                dict(q=None), dict(out=None), dict(batch=dict(n_tok=1 << 24), n_q=16)):
        assert f(**bad) == q8.Q8_0_EINVAL, bad
    for bad in (dict(out=FAKE + 8), dict(q=FAKE + 1), dict(sinks=FAKE + 2), dict(lse=FAKE + 2), dict(ws=FAKE + 8, ws_bytes=64),
                dict(q=FAKE + 2, q_type=0)):
        assert f(**bad) == q8.Q8_0_EALIGN, bad


def test_debug_refusals(q8, calls):
    f = calls["debug"]
    for bad in (dict(kernel=3), dict(kernel=-1), dict(splits=-1), dict(splits=257), dict(kernel=0, splits=2), dict(n_q=7),
                dict(kernel=2, cache=dict(head_dim=512), q_type=0), dict(splits=2, batch=dict(n_tok=1 << 18), n_q=8)):
        assert f(**bad) == q8.Q8_0_EINVAL, bad
    assert f(splits=2, ws=FAKE, ws_bytes=2 * 5 * 8 * 129 * 4 - 1) == q8.Q8_0_EWORKSPACE
    assert f(splits=2) == q8.Q8_0_EWORKSPACE


def test_null_structs(q8):
    lib = q8.raw_library()
    assert lib.kv8_read(None, None, FAKE, FAKE, 1, None) == q8.Q8_0_EINVAL
    assert lib.kv8_attention_workspace_bytes(None, None, 8) == 0


def test_workspace(calls):
    f = calls["workspace"]
    assert f(n_q=7) == 0 and f(n_q=0) == 0 and f(cache=dict(head_dim=96)) == 0 and f(batch=dict(n_seq=0)) == 0
    one = dict(n_seq=1, n_tok=1, max_new=1, table_width=4096)
    # partial outputs and sums of at least two splits for one long sequence, none for a short one
    assert f(batch=one) >= 2 * 8 * 129 * 4
    assert f(batch=dict(one, table_width=1)) == 0
    assert f(batch=dict(one, max_len=64)) == 0


def test_binding_refuses_host_tensors(q8):
    codes, scales = torch.zeros(2, 1, 16, 64, dtype=torch.int8), torch.zeros(2, 1, 1)
    with pytest.raises(ValueError, match="device tensor"):
        q8.Kv8Cache(codes, codes, scales, scales)
    with pytest.raises(ValueError, match="device tensor"):
        q8.Kv8Batch(torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="multiple of block"):
        q8.kv8_cache(1, 1, 64, page_size=64, block=24, device="cpu")


def test_stated_limits(q8, calls):
    """The header's limits of products of sizes: at them a call is looked at further (and refused for its alignment),
    above them refused."""
    wide = dict(batch=dict(n_seq=1, n_tok=1 << 20, max_new=1 << 20), cache=dict(n_kv=1))
    assert calls["attention"](n_q=128, out=FAKE + 8, **wide) == q8.Q8_0_EALIGN
    assert calls["attention"](n_q=129, out=FAKE + 8, **wide) == q8.Q8_0_EINVAL
    for call in ("write", "read"):
        assert calls[call](cache=dict(n_kv=4, k_codes=FAKE + 8), batch=dict(n_seq=1 << 20)) == q8.Q8_0_EALIGN
        assert calls[call](cache=dict(n_kv=5, k_codes=FAKE + 8), batch=dict(n_seq=1 << 20)) == q8.Q8_0_EINVAL
    assert calls["read"](cache=dict(n_pages=1, k_codes=FAKE + 8)) == q8.Q8_0_EALIGN
    assert calls["read"](cache=dict(n_pages=0, k_codes=FAKE + 8)) == q8.Q8_0_EINVAL
