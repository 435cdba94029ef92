"""GPU tests of mxfp4_quantize and mxfp4_dequantize.  The arithmetic of both is
exact, so every comparison is bit for bit."""
import numpy as np
import pytest
import torch

from tests import mxfp4_ref as ref

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def _q8():
    import q8_quantized_matmul_amd as q8
    return q8


def _check(x):
    """Codes, scales and values of the device rows x against the definition."""
    q8 = _q8()
    q = q8.mxfp4_quantize(x)
    codes, scales = ref.quantize(ref.host(x))
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    return q


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,k", [(1, 32), (1, 4096), (3, 96), (37, 1056), (300, 224), (5, 32768)])
def test_rows(rows, k, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows * k)
    x = torch.randn((rows, k), generator=g, device="cuda")
    x = x * torch.exp2(torch.randint(-12, 4, (rows, k // 32, 1), generator=g, device="cuda")
                       .float()).expand(-1, -1, 32).reshape(rows, k)
    _check(x.to(dtype))


@pytest.mark.parametrize("dtype", DTYPES)
def test_every_binade_ties_and_neighbours(dtype):
    """Each rounding boundary, its neighbours and its negatives, with the block
    maximum in every binade of the type, subnormals included."""
    top = {torch.float32: 127, torch.bfloat16: 127, torch.float16: 15}[dtype]
    low = {torch.float32: -149, torch.bfloat16: -133, torch.float16: -24}[dtype]
    marks = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 1.0, 6.0])
    eps = float(torch.finfo(dtype).eps)
    near = np.concatenate([marks, marks * (1 - eps), marks * (1 + eps)])
    rows = []
    for e in range(low, top + 1):
        block = np.zeros(32)
        block[0] = 1.5 * 2.0 ** e        # the maximum: scale 2^(e-2) where that exists
        block[1:31] = near * 2.0 ** (e - 2) * np.where(np.arange(30) % 3 == 0, -1, 1)
        rows.append(np.where(np.abs(block) < 1.9 * 2.0 ** e, block, 0.0))
    x = torch.from_numpy(np.array(rows)).to(dtype).cuda()
    assert torch.isfinite(x).all()
    _check(x)


@pytest.mark.parametrize("dtype", DTYPES)
def test_special_blocks(dtype):
    """A NaN or infinity poisons its own block only; zero blocks keep signs;
    the largest finite values are held at 6 * 2^E."""
    x = torch.zeros((8, 64), dtype=dtype, device="cuda")
    x[0, 3] = float("nan")
    x[1, 40] = float("inf")
    x[2, 0] = -float("inf")
    x[3] = -0.0
    x[4, :32] = torch.finfo(dtype).max
    x[5, 7] = torch.finfo(dtype).smallest_normal
    x[6] = -torch.finfo(dtype).tiny
    x[7, 63] = 1.0
    q = _check(x)
    s = q.scales.cpu().numpy()
    assert s[0].tolist() == [255, 0] and s[1].tolist() == [0, 255] and s[3].tolist() == [0, 0]
    v = _q8().mxfp4_dequantize(q)
    assert torch.isnan(v[0, :32]).all() and (v[0, 32:] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad,shift", [(32, 0), (8, 8), (1, 0), (3, 1), (96, 5)])
def test_row_stride_and_alignment(dtype, pad, shift):
    """Rows cut out of a wider tensor, starting at any element; the outputs'
    surroundings stay as they were."""
    q8 = _q8()
    rows, k = 19, 160
    wide = torch.randn((rows, k + pad + shift), device="cuda").to(dtype)
    x = wide[:, shift:shift + k]
    codes = torch.full((rows + 2, k // 2), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows + 2, k // 32), 0xA5, dtype=torch.uint8, device="cuda")
    q8.mxfp4_quantize(x, codes=codes[1:-1], scales=scales[1:-1])
    want = ref.quantize(ref.host(x))
    assert np.array_equal(codes[1:-1].cpu().numpy(), want[0])
    assert np.array_equal(scales[1:-1].cpu().numpy(), want[1])
    for t in (codes, scales):
        assert (t[0] == 0xA5).all() and (t[-1] == 0xA5).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_dequantize_every_code_and_scale(dtype):
    q8 = _q8()
    codes = np.tile(np.arange(256, dtype=np.uint8).reshape(16, 16), (256, 1))
    scales = np.repeat(np.arange(256, dtype=np.uint8), 16)[:, None]
    got = q8.mxfp4_dequantize(ref.device(q8, (codes, scales)), dtype=dtype)
    want = torch.from_numpy(ref.values(codes, scales)).to(dtype)  # one rounding, exact but for fp16
    got, nan = got.cpu(), torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("shape", [(1, 32), (7, 96), (3, 5, 64), (2, 8192)])
def test_dequantize_shapes(shape):
    q8 = _q8()
    m = ref.random_matrix(np.random.default_rng(3), shape)
    got = q8.mxfp4_dequantize(ref.device(q8, m), dtype=torch.bfloat16)
    assert tuple(got.shape) == shape
    assert np.array_equal(ref.host(got), ref.values(*m))


def test_offsets_beyond_32_bits():
    """Rows whose first element lies past 2^32 bytes."""
    q8 = _q8()
    k, rows, stride = 64, 3, 1_500_000_000
    x = torch.empty(stride * (rows - 1) + k, dtype=torch.bfloat16, device="cuda")
    view = torch.as_strided(x, (rows, k), (stride, 1))
    view.copy_(torch.randn((rows, k), device="cuda"))
    q = q8.mxfp4_quantize(view)
    want = ref.quantize(ref.host(view))
    assert np.array_equal(q.codes.cpu().numpy(), want[0])
    assert np.array_equal(q.scales.cpu().numpy(), want[1])


def test_empty_and_other_stream():
    q8 = _q8()
    assert q8.mxfp4_quantize(torch.empty((0, 64), device="cuda")).codes.shape == (0, 32)
    s = torch.cuda.Stream()
    x = torch.randn((64, 256), device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        q = q8.mxfp4_quantize(x)
        v = q8.mxfp4_dequantize(q)
    s.synchronize()
    assert np.array_equal(ref.host(v), ref.values(*ref.quantize(ref.host(x))))
