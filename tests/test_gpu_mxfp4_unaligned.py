"""Scale arrays at any byte give the very bits that aligned ones do: neither the plan
nor the order of the sums depends on where they lie.  Streaming and tiled kernels, each
tile, with rows of a block count that is and is not a multiple of sixteen."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _at(m, shift):
    """The matrix with its scales `shift` bytes into a buffer, between bytes of 255."""
    import q8_quantized_matmul_amd as q8
    buf = torch.full((m.scales.numel() + 32,), 255, dtype=torch.uint8, device="cuda")
    s = buf[shift:shift + m.scales.numel()].view(m.scales.shape)
    s.copy_(m.scales)
    return q8.Mxfp4(m.codes, s)


@pytest.mark.parametrize("k,n,t", [
    (1024, 64, 3), (1056, 64, 20), (32800, 200, 1),            # streaming
    (1024, 300, 200), (1056, 300, 200), (544, 1000, 40),       # 64 x 64 tiles
    (4128, 4096, 1024), (4128, 2048, 2048), (4128, 4096, 2048),
    (4128, 2048, 4096), (32800, 1024, 2048), (4096, 4096, 4096), (4128, 4096, 4096),
])
def test_matmul(k, n, t):
    import q8_quantized_matmul_amd as q8
    g = torch.Generator(device="cuda").manual_seed(k + n + t)
    w, x = (q8.Mxfp4(torch.randint(0, 256, (r, k // 2), dtype=torch.uint8, device="cuda", generator=g),
                     torch.randint(118, 124, (r, k // 32), dtype=torch.uint8, device="cuda", generator=g)) for r in (n, t))
    base = q8.mxfp4_matmul(w, x)
    assert torch.isfinite(base).all()
    for a, b in ((1, 0), (0, 1), (3, 2), (15, 7)):
        assert torch.equal(q8.mxfp4_matmul(_at(w, a), _at(x, b)), base), (a, b)
