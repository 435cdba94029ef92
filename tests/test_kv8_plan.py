"""CPU checks of the plan that kv8_attention takes for a workspace: what it makes the kernels
write fits, to the byte."""
import ctypes

import pytest


class Cache(ctypes.Structure):
    """kv::Cache of kv8_launch.h."""
    _fields_ = [("pointers", ctypes.c_void_p * 4), ("n_pages", ctypes.c_int32), ("n_kv", ctypes.c_int32),
                ("d", ctypes.c_int32), ("page_log", ctypes.c_int), ("block_log", ctypes.c_int)]


class Batch(ctypes.Structure):
    """kv::Batch."""
    _fields_ = [("pointers", ctypes.c_void_p * 3), ("n_seq", ctypes.c_int32), ("n_tok", ctypes.c_int32),
                ("width", ctypes.c_int32), ("max_new", ctypes.c_int32), ("max_len", ctypes.c_int32)]


class Plan(ctypes.Structure):
    """kv::Plan."""
    _fields_ = [("tiled", ctypes.c_bool), ("splits", ctypes.c_int)]


@pytest.fixture(scope="module")
def plan():
    import q8_quantized_matmul_amd as q8
    f = getattr(ctypes.CDLL(q8.LIB_PATH), "_ZN2kv14attention_planERKNS_5CacheERKNS_5BatchEiibm")
    f.argtypes = [ctypes.POINTER(Cache), ctypes.POINTER(Batch), ctypes.c_int, ctypes.c_int, ctypes.c_bool, ctypes.c_size_t]
    f.restype = Plan

    def call(c, b, n_q, window, halves, ws_bytes):
        p = f(ctypes.byref(c), ctypes.byref(b), n_q, window, halves, ws_bytes)
        return p.tiled, p.splits
    return call


def bytes_of(d, n_tok, n_q, splits):
    return splits * n_tok * n_q * (d + 1) * 4 if splits > 1 else 0


# (sequences, rows of each, query heads, key/value heads, head size, longest): most fastest plans have partial
# results above 2^24 bytes, where fp32 does not hold every number of bytes (185 270 272 for the first)
LARGE = [(16, 8, 64, 8, 256, 524288), (8, 8, 64, 8, 256, 524288), (64, 1, 32, 1, 512, 131072), (1, 512, 32, 8, 128, 65536),
         (1, 600, 64, 1, 512, 100000), (3, 37, 40, 8, 192, 300000), (1, 1024, 128, 8, 64, 262144)]


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("window", [0, 50000])
@pytest.mark.parametrize("sizes", LARGE)
def test_plan_fits_the_workspace(plan, sizes, window, halves):
    n_seq, new, n_q, n_kv, d, longest = sizes
    c = Cache(n_pages=1 << 20, n_kv=n_kv, d=d, page_log=8, block_log=4)
    b = Batch(n_seq=n_seq, n_tok=n_seq * new, width=longest >> 8, max_new=new, max_len=longest)
    kind, splits = plan(c, b, n_q, window, halves, 2 ** 64 - 1)
    need = bytes_of(d, n_seq * new, n_q, splits)
    assert plan(c, b, n_q, window, halves, need) == (kind, splits)
    for less in (1, 4, 8, 16, 64, 256, 4096):
        ws = max(need - less, 0)
        _, fewer = plan(c, b, n_q, window, halves, ws)
        assert bytes_of(d, n_seq * new, n_q, fewer) <= ws
    assert plan(c, b, n_q, window, halves, 0)[1] == 1
