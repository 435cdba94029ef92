"""GPU tests of what include/mxfp4.h says of moe_topk's keys and of infinite scores."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _topk(*args, **kw):
    import q8_quantized_matmul_amd as q8
    return q8.moe_topk(*args, **kw)


@pytest.mark.parametrize("e", [40, 300])
def test_a_softmax_bias_is_added_to_the_logits(e):
    """The order of probability * exp(bias), in 64 bits where no two keys are nearly
    equal, and not that of probability + bias."""
    g = torch.Generator(device="cuda").manual_seed(e)
    z = torch.randn((50, e), generator=g, device="cuda")
    b = torch.randn((e,), generator=g, device="cuda") * 0.5
    sel, w = _topk(z, 4, bias=b)
    p = torch.softmax(z.double(), -1)
    key = (p * torch.exp(b.double())).sort(-1, descending=True)
    gap = key.values[:, :4] / key.values[:, 1:5] - 1
    clear = (gap > 1e-5).all(1)  # an fp32 sum of numbers below 8 is off by 2^-22 at most
    assert clear.float().mean() > 0.9
    assert torch.equal(sel[clear].long(), key.indices[clear, :4])
    added = (p + b.double()).topk(4).indices
    assert not torch.equal(sel[clear].long(), added[clear])
    chosen = torch.gather(p, 1, sel.long())
    want = chosen / chosen.sum(-1, keepdim=True)
    np.testing.assert_allclose(w.cpu().numpy(), want.cpu().numpy(), rtol=(8 + 16 + 30) * 2.0 ** -24)


@pytest.mark.parametrize("e", [40, 300])
def test_an_infinite_score(e):
    z = torch.randn((3, e), device="cuda")
    z[1, 7] = float("inf")
    _, w = _topk(z, 4, scoring=0)
    assert torch.isnan(w[1]).all() and torch.isfinite(w[[0, 2]]).all()
    sel, w = _topk(z, 4, scoring=2)
    assert sel[1, 0] == 7 and torch.isnan(w[1, 0]) and (w[1, 1:] == 0).all() and torch.isfinite(w[[0, 2]]).all()
    _, w = _topk(z, 4, scoring=2, renormalize=False)
    assert torch.isposinf(w[1, 0]) and torch.isfinite(w[1, 1:]).all()
    _, w = _topk(z, 4, scoring=1)
    assert torch.isfinite(w).all()
