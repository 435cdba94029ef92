"""Matrices whose bytes, and outputs whose elements, do not fit 32-bit offsets.

Codes at scale 1 give sums that fp32 holds exactly (products are multiples of
1/4, at most 36 each), so equality does not depend on the order of summation."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _q8():
    import q8_quantized_matmul_amd as q8
    return q8


def _mat(*shape, scale=127):
    *lead, k = shape
    return _q8().Mxfp4(torch.randint(0, 256, (*lead, k // 2), dtype=torch.uint8, device="cuda"),
                       torch.full((*lead, k // 32), scale, dtype=torch.uint8, device="cuda"))


def _rows(m, a, b):
    return _q8().Mxfp4(m.codes[a:b].contiguous(), m.scales[a:b].contiguous())


def _product(x, w):
    q8 = _q8()
    return q8.mxfp4_dequantize(x).double() @ q8.mxfp4_dequantize(w).double().t().contiguous()


@pytest.mark.parametrize("t", [1, 24, 100])
def test_weights_beyond_32_bits(t):
    q8 = _q8()
    n, k = 280000, 32768
    assert n * k // 2 > 2 ** 32 and k * 36 * 4 < 2 ** 24
    w, x = _mat(n, k), _mat(t, k)
    out = q8.mxfp4_matmul(w, x)
    for a in (0, 262140, n - 48):  # the first, those around byte 2^32, the last
        assert torch.equal(out[:, a:a + 48].double(), _product(x, _rows(w, a, a + 48))), a


@pytest.mark.parametrize("k,n,t", [(512, 32768, 70001), (32, 32768, 70001)])
def test_output_beyond_32_bits(k, n, t):
    q8 = _q8()
    assert n * t > 2 ** 31
    w, x = _mat(n, k), _mat(t, k)
    out = q8.mxfp4_matmul(w, x)
    for a in (0, 65520, t - 33):
        assert torch.equal(out[a:a + 33].double(), _product(_rows(x, a, a + 33), w)), a


@pytest.mark.parametrize("t", [1, 9])
def test_experts_beyond_32_bits(t):
    """Four experts at both ends of 300 give what a layer of those four gives: the
    same ids and weights, and outputs that differ by the order of their sum at most
    (a token alone adds its experts by score, others by id)."""
    q8 = _q8()
    torch.manual_seed(t)
    e, d, f, ids = 300, 8192, 4096, [0, 260, 298, 299]
    assert e * d * f // 2 > 2 ** 32
    mats = [_mat(e, *shape, scale=116) for shape in ((f, d), (f, d), (d, f))]
    small = [q8.Mxfp4(m.codes[ids].contiguous(), m.scales[ids].contiguous()) for m in mats]
    index = torch.tensor(ids, dtype=torch.int32, device="cuda")
    for _ in range(4):
        x = torch.randn((t, d), device="cuda")
        z = torch.full((t, e), -float("inf"), device="cuda")
        few = torch.randn((t, 4), device="cuda")
        z[:, ids] = few
        out, sel, w = q8.mxfp4_moe_layer(x, z, *mats, 3)
        out4, sel4, w4 = q8.mxfp4_moe_layer(x, few, *small, 3)
        assert torch.isfinite(out).all() and out.abs().max() > 0
        assert torch.equal(sel, index[sel4.long()]) and torch.equal(w, w4)
        # Each expert alone, with weight 1.  The three products w_j y_j are the same in
        # both sums, and each sum's two additions round by at most 2^-24 of the sum of
        # the magnitudes: four such steps lie between the two.
        alone = []
        for j in range(4):
            only = torch.full((t, 4), -float("inf"), device="cuda")
            only[:, j] = 0.0
            alone.append(q8.mxfp4_moe_layer(x, only, *small, 1)[0].double().abs())
        y = torch.stack(alone, 1)  # [t][4][d]
        total = sum(w4[:, j, None].double() * y[torch.arange(t), sel4[:, j].long()] for j in range(3))
        assert ((out.double() - out4.double()).abs() <= 4.01 * 2.0 ** -24 * total).all()


def test_quantizer_beyond_32_bits():
    """More than 2^32 values, so more workgroups than the grid has along x: every slice
    equals the slice's own result, and the bytes behind the end stay as they were."""
    q8 = _q8()
    rows, k = 131075, 32768
    assert rows * k > 2 ** 32
    x = torch.randn((rows, k), dtype=torch.bfloat16, device="cuda")
    codes = torch.full((rows + 1, k // 2), 77, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows + 1, k // 32), 77, dtype=torch.uint8, device="cuda")
    q8.mxfp4_quantize(x, codes=codes[:rows], scales=scales[:rows])
    back = q8.mxfp4_dequantize(q8.Mxfp4(codes[:rows], scales[:rows]), torch.bfloat16)
    for a in (0, 65534, 131070):  # the first, those around values 2^31 and 2^32
        q = q8.mxfp4_quantize(x[a:a + 5])
        assert torch.equal(codes[a:a + 5], q.codes) and torch.equal(scales[a:a + 5], q.scales), a
        assert torch.equal(back[a:a + 5], q8.mxfp4_dequantize(q, torch.bfloat16)), a
    assert (codes[rows] == 77).all() and (scales[rows] == 77).all()
