"""Sizes that do not fit the C calls' 32-bit arguments are refused by the binding, and
never taken for their low 32 bits."""
import pytest
import torch

BEYOND = 2 ** 32 + 4  # the low 32 bits are a valid size


def _q8():
    import q8_quantized_matmul_amd as q8
    return q8


def test_layer_workspace():
    q8 = _q8()
    assert q8.mxfp4_moe_layer_workspace_bytes(8, 4, 16, 256, 128) > 0
    with pytest.raises(ValueError):
        q8.mxfp4_moe_layer_workspace_bytes(8, BEYOND, 16, 256, 128)
    with pytest.raises(ValueError):
        q8.mxfp4_moe_layer_workspace_bytes(8, 4, BEYOND, 256, 128)


@pytest.mark.gpu
def test_router():
    q8 = _q8()
    z = torch.randn((2, 16), device="cuda")
    with pytest.raises(ValueError):
        q8.moe_topk(z, BEYOND)
    with pytest.raises(ValueError):
        q8.moe_topk(z, 2, scoring=2 ** 32 + 1)
    with pytest.raises(ValueError):
        q8.moe_topk(torch.empty((1, BEYOND), device="cuda"), 2)


@pytest.mark.gpu
def test_layer():
    q8 = _q8()
    mat = lambda *s: q8.Mxfp4(torch.zeros((*s[:-1], s[-1] // 2), dtype=torch.uint8, device="cuda"),
                              torch.zeros((*s[:-1], s[-1] // 32), dtype=torch.uint8, device="cuda"))
    args = (torch.zeros((2, 64), device="cuda"), torch.zeros((2, 16), device="cuda"), mat(16, 32, 64), mat(16, 32, 64), mat(16, 64, 32))
    q8.mxfp4_moe_layer(*args, 4)
    with pytest.raises(ValueError):
        q8.mxfp4_moe_layer(*args, BEYOND)
    with pytest.raises(ValueError):
        q8.mxfp4_moe_layer(*args, 4, scoring=2 ** 32)
