"""GPU tests of mxfp4_matmul, and of mxfp4_dequantize, at both ends of the scale range, against 64 bits.

A block's values reach from 2^-128 to 6 * 2^127, so the terms of a product leave
fp32's normal numbers on both sides.  Below 2^-126 a term, or one of the at most
k / 32 + 8 rounded sums, may lose its fraction or all of itself, 2^-126 at most: with
k terms that is less than k * 2^-125 together (k / 32 + 8 <= k), beside the (k / 32 +
8) steps of 2^-23 of sum |w x|.  Above 2^128 a term or a partial sum is infinite, and
infinities of both signs make a NaN; where sum |w x| lies below 2^127 no partial sum
in any order does."""
import numpy as np
import pytest
import torch

from tests import mxfp4_ref as ref

pytestmark = pytest.mark.gpu

# Streaming, streaming split over workgroups, and the tiles of the tiled kernel.
SHAPES = [(96, 40, 5), (1024, 64, 3), (32768, 256, 1), (1056, 64, 40), (1024, 256, 300), (1056, 2048, 2048), (4096, 4096, 4096)]


def _product(w, x):
    """(out [t][n] as the call gives it, exact, sum |w x|) of some tokens."""
    import q8_quantized_matmul_amd as q8
    out = q8.mxfp4_matmul(ref.device(q8, w), ref.device(q8, x))
    rows = sorted({0, len(x[0]) // 2, len(x[0]) - 1})
    wv, xv = ref.values(*w), ref.values(*x)[rows]
    return ref.host(out)[rows], xv @ wv.T, np.abs(xv) @ np.abs(wv).T


def _bound(k, mag):
    return (k / 32 + 8) * 2.0 ** -23 * mag + k * 2.0 ** -125


@pytest.mark.parametrize("w_bytes,x_bytes", [((0, 20), (0, 20)), ((60, 66), (60, 66)), ((40, 60), (60, 66)), ((0, 8), (118, 126))])
@pytest.mark.parametrize("k,n,t", SHAPES)
def test_terms_below_the_normal_numbers(k, n, t, w_bytes, x_bytes):
    rng = np.random.default_rng([k, n, t, *w_bytes])
    got, want, mag = _product(ref.random_matrix(rng, (n, k), *w_bytes), ref.random_matrix(rng, (t, k), *x_bytes))
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= _bound(k, mag)).all()


@pytest.mark.parametrize("k,n,t", SHAPES)
def test_terms_above_the_largest_number(k, n, t):
    """Ordinary rows and rows whose products overflow, among tokens of both kinds: an
    overflow stays with its output, which is then never finite."""
    rng = np.random.default_rng([k, n, t, 1])
    w, x = ref.random_matrix(rng, (n, k), 120, 126), ref.random_matrix(rng, (t, k), 120, 126)
    w[1][n // 2:] = rng.integers(186, 255, w[1][n // 2:].shape)
    if t > 1:
        x[1][t - 1] = rng.integers(186, 255, k // 32)
    w[0][n - 1] &= 0x77  # a row and a token without signs
    x[0][t - 1] &= 0x77
    got, want, mag = _product(w, x)
    finite = np.isfinite(got)
    small, large = mag < 2.0 ** 127, np.abs(want) - _bound(k, mag) >= 2.0 ** 128
    assert small.any() and large.any() and large[-1, n - 1]
    assert finite[small].all() and not finite[large].any()
    assert (np.abs(got - want) <= _bound(k, mag))[finite].all()
    assert np.isposinf(got[-1, n - 1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_largest_scales_dequantized(dtype):
    """Exact below 2^128 and infinite from there on; what the quantizer makes of the
    largest numbers is below."""
    import q8_quantized_matmul_amd as q8
    codes = np.tile(np.arange(256, dtype=np.uint8).reshape(16, 16), (3, 1))
    scales = np.repeat(np.array([252, 253, 254], dtype=np.uint8), 16)[:, None]
    got, want = ref.host(q8.mxfp4_dequantize(ref.device(q8, (codes, scales)), dtype)), ref.values(codes, scales)
    large = np.abs(want) >= 2.0 ** 128
    assert large[16:].any() and not large[:16].any()
    assert np.array_equal(got, np.where(large, np.copysign(np.inf, want), want))
    x = torch.full((2, 64), torch.finfo(dtype).max, dtype=dtype, device="cuda")
    x[1] = -x[1]
    q = q8.mxfp4_quantize(x)
    assert (q.scales == 252).all()
    assert torch.equal(q8.mxfp4_dequantize(q, dtype), torch.sign(x) * 6 * 2.0 ** 125)
