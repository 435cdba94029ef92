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


def test_matmul_refusals(q8, lib):
    def call(out=FAKE, out_type=0, wc=FAKE, ws=FAKE, k=64, n=16, xc=FAKE, xs=FAKE, t=2, work=None, nbytes=0):
        return lib.mxfp4_matmul(out, out_type, wc, ws, k, n, xc, xs, t, work, nbytes, None)
    assert call(k=48) == q8.Q8_0_EINVAL
    assert call(k=0) == q8.Q8_0_EINVAL
    assert call(k=(1 << 24) + 32) == q8.Q8_0_EINVAL
    assert call(n=-1) == q8.Q8_0_EINVAL
    assert call(t=(1 << 30) + 1) == q8.Q8_0_EINVAL
    assert call(n=1 << 20, t=1 << 19) == q8.Q8_0_EINVAL
    assert call(out_type=7) == q8.Q8_0_EINVAL
    for name in ("out", "wc", "ws", "xc", "xs"):
        assert call(**{name: None}) == q8.Q8_0_EINVAL
    assert call(wc=FAKE + 8) == q8.Q8_0_EALIGN
    assert call(xc=FAKE + 4) == q8.Q8_0_EALIGN
    assert call(out=FAKE + 2) == q8.Q8_0_EALIGN
    assert call(out=FAKE + 1, out_type=1) == q8.Q8_0_EALIGN
    assert call(work=FAKE + 8, nbytes=64) == q8.Q8_0_EALIGN
    assert call(t=0) == q8.Q8_0_OK
    assert call(n=0) == q8.Q8_0_OK


def test_matmul_workspace(q8):
    """Only long rows with too few tiles to fill the chip split, into whole partial outputs."""
    size = q8.mxfp4_matmul_workspace_bytes
    for k, n, t in ((4096, 2048, 1), (4096, 4096, 4096), (96, 64, 200), (64, 0, 100), (64, 64, 0), (33, 64, 64)):
        assert size(k, n, t) == 0, (k, n, t)
    assert size(32768, 1024, 2048) == 4 * 1024 * 2048 * 4
    for k, n, t in ((16384, 512, 100), (32768, 1024, 1), (32768, 40, 20)):
        need = size(k, n, t)
        assert need > 0 and need % (n * t * 4) == 0, (k, n, t)


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


def test_layer_refusals(q8, lib):
    need = q8.mxfp4_moe_layer_workspace_bytes(8, 4, 16, 256, 128)
    assert need >= 8 * 4 * (64 + 4)

    def call(ws=FAKE, ws_bytes=need, **kw):
        f = dict(out=FAKE, x=FAKE, out_type=1, x_type=1, logits=FAKE, bias=None, n_expert=16, n_used=4,
                 scoring=0, renormalize=1, scale=1.0, clamp=0.0, d_model=256, d_ff=128, n_tok=8,
                 gate_codes=FAKE, gate_scales=FAKE, up_codes=FAKE, up_scales=FAKE, down_codes=FAKE,
                 down_scales=FAKE, selected=None, weights=None)
        f.update(kw)
        return lib.mxfp4_moe_layer(ctypes.byref(q8.MoeLayerArgs(**f)), ws, ws_bytes, None)

    assert lib.mxfp4_moe_layer(None, FAKE, need, None) == q8.Q8_0_EINVAL
    for bad in (dict(n_tok=65), dict(n_tok=-1), dict(n_expert=0), dict(n_expert=513), dict(n_used=0),
                dict(n_used=17), dict(d_model=100), dict(d_model=0), dict(d_ff=48), dict(d_ff=1 << 21),
                dict(scoring=3), dict(x_type=3), dict(out_type=-1), dict(n_expert=512, d_model=1 << 20, d_ff=1 << 20)):
        assert call(**bad) == q8.Q8_0_EINVAL, bad
    for name in ("out", "x", "logits", "gate_codes", "gate_scales", "up_codes", "up_scales", "down_codes", "down_scales"):
        assert call(**{name: None}) == q8.Q8_0_EINVAL, name
    for name in ("out", "x", "gate_codes", "up_codes", "down_codes"):
        assert call(**{name: FAKE + 8}) == q8.Q8_0_EALIGN, name
    for name in ("logits", "bias", "selected", "weights"):
        assert call(**{name: FAKE + 2}) == q8.Q8_0_EALIGN, name
    assert call(ws=None) == q8.Q8_0_EWORKSPACE
    assert call(ws_bytes=need - 1) == q8.Q8_0_EWORKSPACE
    assert call(ws=FAKE + 64) == q8.Q8_0_EALIGN
    assert call(n_tok=0) == q8.Q8_0_OK
    assert q8.mxfp4_moe_layer_workspace_bytes(65, 4, 16, 256, 128) == 0
    if torch.cuda.device_count() == 0:
        assert call() == q8.Q8_0_ENODEV


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
    assert lib.mxfp4_matmul(FAKE, 0, FAKE, FAKE, 64, 16, FAKE, FAKE, 2, None, 0, None) == q8.Q8_0_ENODEV


def test_sizes_at_the_limits(q8, lib):
    """The largest sizes pass the checks (and find no device), one more does not."""
    if torch.cuda.device_count() > 0:
        pytest.skip("a device is present")

    def mm(k, n, t):
        return lib.mxfp4_matmul(FAKE, 1, FAKE, FAKE, k, n, FAKE, FAKE, t, None, 0, None)
    assert mm(1 << 24, 1 << 28, 128) == mm(32, 128, 1 << 28) == q8.Q8_0_ENODEV
    assert mm((1 << 24) + 32, 1, 1) == mm(32, (1 << 28) + 1, 1) == mm(32, 1, (1 << 28) + 1) == q8.Q8_0_EINVAL
    assert mm(32, 1 << 28, 129) == q8.Q8_0_EINVAL

    def topk(t):
        return lib.moe_topk(FAKE, FAKE, FAKE, None, t, 8, 2, 0, 1, 1.0, None)
    assert topk(1 << 25) == q8.Q8_0_ENODEV and topk((1 << 25) + 1) == q8.Q8_0_EINVAL
    assert lib.mxfp4_quantize(FAKE, FAKE, FAKE, 1, 1 << 20, 1 << 23, 1 << 20, None) == q8.Q8_0_ENODEV
    assert lib.mxfp4_quantize(FAKE, FAKE, FAKE, 1, 1 << 20, (1 << 23) + 1, 1 << 20, None) == q8.Q8_0_EINVAL
