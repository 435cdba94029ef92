"""CPU checks of include/mxfp4.h: every declared function is exported and bound,
and the host-side argument checks refuse what the header says they refuse.
No call here reaches a device: each fails validation, or is empty."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def q8():
    import q8_quantized_matmul_amd as m
    return m


@pytest.fixture(scope="module")
def lib(q8):
    return q8.raw_library()


def test_exports_every_declared_symbol(q8):
    from q8_quantized_matmul_amd import mxfp4
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mxfp4.h")).read(), flags=re.S)
    declared = set(re.findall(r"\b((?:mxfp4|moe)_\w+)\s*\(", text))
    assert declared == set(mxfp4.EXPORTED)
    lib = ctypes.CDLL(q8.LIB_PATH)
    for name in declared:
        assert hasattr(lib, name) and (name.endswith("_bytes") or hasattr(q8, name)), name


def test_quantize_refusals(q8, lib):
    def call(codes=FAKE, scales=FAKE, x=FAKE, x_type=0, stride=64, rows=2, k=64):
        return lib.mxfp4_quantize(codes, scales, x, x_type, stride, rows, k, None)
    assert call(k=33) == q8.Q8_0_EINVAL
    assert call(rows=-1) == q8.Q8_0_EINVAL
    assert call(stride=63) == q8.Q8_0_EINVAL
    assert call(x_type=3) == q8.Q8_0_EINVAL
    assert call(rows=1 << 60, k=1 << 20, stride=1 << 20) == q8.Q8_0_EINVAL
    for name in ("codes", "scales", "x"):
        assert call(**{name: None}) == q8.Q8_0_EINVAL
    assert call(codes=FAKE + 8) == q8.Q8_0_EALIGN
    assert call(x=FAKE + 2) == q8.Q8_0_EALIGN
    assert call(x=FAKE + 1, x_type=1) == q8.Q8_0_EALIGN
    assert call(rows=0) == q8.Q8_0_OK
    assert call(k=0) == q8.Q8_0_OK


def test_dequantize_refusals(q8, lib):
    def call(out=FAKE, out_type=0, codes=FAKE, scales=FAKE, rows=2, k=64):
        return lib.mxfp4_dequantize(out, out_type, codes, scales, rows, k, None)
    assert call(k=16) == q8.Q8_0_EINVAL
    assert call(rows=-1) == q8.Q8_0_EINVAL
    assert call(out_type=-1) == q8.Q8_0_EINVAL
    for name in ("codes", "scales", "out"):
        assert call(**{name: None}) == q8.Q8_0_EINVAL
    assert call(out=FAKE + 8) == q8.Q8_0_EALIGN
    assert call(codes=FAKE + 4) == q8.Q8_0_EALIGN
    assert call(rows=0) == q8.Q8_0_OK


def test_topk_refusals(q8, lib):
    def call(sel=FAKE, w=FAKE, logits=FAKE, bias=None, t=4, e=256, u=8, scoring=0):
        return lib.moe_topk(sel, w, logits, bias, t, e, u, scoring, 1, 1.0, None)
    assert call(e=0) == q8.Q8_0_EINVAL
    assert call(e=1025) == q8.Q8_0_EINVAL
    assert call(u=0) == q8.Q8_0_EINVAL
    assert call(u=33) == q8.Q8_0_EINVAL
    assert call(e=4, u=5) == q8.Q8_0_EINVAL
    assert call(scoring=3) == q8.Q8_0_EINVAL
    assert call(t=-1) == q8.Q8_0_EINVAL
    assert call(t=1 << 29) == q8.Q8_0_EINVAL
    for name in ("sel", "w", "logits"):
        assert call(**{name: None}) == q8.Q8_0_EINVAL
        assert call(**{name: FAKE + 2}) == q8.Q8_0_EALIGN
    assert call(bias=FAKE + 1) == q8.Q8_0_EALIGN
    assert call(t=0) == q8.Q8_0_OK


def test_binding_refuses_host_tensors_and_wrong_shapes(q8):
    with pytest.raises(ValueError):
        q8.mxfp4_quantize(torch.zeros(2, 64))
    with pytest.raises(ValueError):
        q8.mxfp4_quantize(torch.zeros(2, 2, 64))
    with pytest.raises(ValueError):
        q8.mxfp4_dequantize(q8.Mxfp4(torch.zeros(2, 32, dtype=torch.uint8),
                                     torch.zeros(2, 2, dtype=torch.uint8)))


def test_valid_calls_without_device_report_nodev(q8, lib):
    if torch.cuda.device_count() > 0:
        pytest.skip("a device is present")
    assert lib.mxfp4_quantize(FAKE, FAKE, FAKE, 0, 64, 2, 64, None) == q8.Q8_0_ENODEV
    assert lib.mxfp4_dequantize(FAKE, 0, FAKE, FAKE, 2, 64, None) == q8.Q8_0_ENODEV
    assert lib.moe_topk(FAKE, FAKE, FAKE, None, 4, 256, 8, 0, 1, 1.0, None) == q8.Q8_0_ENODEV
