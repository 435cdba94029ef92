"""The MXFP4 calls after the LDS of every compute unit was filled with a pattern
(as the Q8_0 calls' tests do): every run equals the first bit for bit, so no
kernel reads LDS before it is written, or before the barrier that publishes
another wave's writes.  Each size takes another kernel or another split."""
import pytest
import torch

pytestmark = pytest.mark.gpu

PATTERNS = [0x00000000, 0xFFFFFFFF, 0x7F7F7F7F, 0x80000001]


def _q8():
    import q8_quantized_matmul_amd as q8
    return q8


def _mat(g, *shape):
    q8 = _q8()
    *lead, k = shape
    return q8.Mxfp4(torch.randint(0, 256, (*lead, k // 2), dtype=torch.uint8, device="cuda", generator=g),
                    torch.randint(118, 122, (*lead, k // 32), dtype=torch.uint8, device="cuda", generator=g))


def _same_after_every_pattern(call):
    first = [o.clone() for o in call()]
    for o in first:
        assert not torch.isnan(o.float()).any()
    for pattern in PATTERNS:
        _q8().q8_0_debug_poison_lds(pattern)
        for a, b in zip(first, call()):
            assert torch.equal(a, b), hex(pattern)


@pytest.mark.parametrize("k,n,t", [
    (1024, 4096, 1), (32768, 256, 1), (2912, 1000, 13), (96, 50, 40),         # streaming, split and ragged
    (4096, 2048, 200), (1056, 320, 70), (7168, 512, 129),                     # 64x64 tiles, odd, split
    (4096, 2048, 2048), (4096, 2048, 4000), (4096, 4096, 4096), (8224, 1000, 2000),
])
def test_matmul(k, n, t):
    q8 = _q8()
    g = torch.Generator(device="cuda").manual_seed(k + n + t)
    w, x = _mat(g, n, k), _mat(g, t, k)
    _same_after_every_pattern(lambda: [q8.mxfp4_matmul(w, x)])


@pytest.mark.parametrize("t,d,f,e,u", [(1, 1024, 256, 16, 4), (8, 544, 96, 20, 3), (11, 1056, 352, 20, 4),
                                       (64, 256, 128, 300, 8), (3, 64, 64, 4, 2)])
def test_moe_layer(t, d, f, e, u):
    q8 = _q8()
    g = torch.Generator(device="cuda").manual_seed(t * d + f)
    mats = _mat(g, e, f, d), _mat(g, e, f, d), _mat(g, e, d, f)
    x = torch.randn((t, d), generator=g, device="cuda")
    z = torch.randn((t, e), generator=g, device="cuda")
    for scoring in (0, 1):
        _same_after_every_pattern(lambda: q8.mxfp4_moe_layer(x, z, *mats, u, scoring=scoring))
