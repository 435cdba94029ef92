"""GPU tests of what include/mxfp4.h says of moe_topk's keys and of infinite scores."""
import numpy as np
import pytest
import torch

from tests import mxfp4_ref as ref

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


@pytest.mark.parametrize("scoring", [1, 2])
@pytest.mark.parametrize("t,e,u", [(1, 1, 1), (40, 9, 1), (50, 14, 11), (30, 64, 8), (50, 200, 4), (20, 1024, 32)])
def test_scores_below_the_range_of_fp32(t, e, u, scoring):
    """Logits of -60 to -700, alone and beside ordinary ones, renormalized: scores of
    which fp32 holds a few bits or none still give weights that sum to one.  A weight
    carries a rounding of its score, at most 24 of the sum and the division and scale:
    as in test_gpu_moe_topk, 29 half steps; 2^-126 where it is subnormal itself."""
    g = torch.Generator(device="cuda").manual_seed(t * e + u + scoring)
    far = -60 - 640 * torch.rand((t, 1), generator=g, device="cuda")
    z = far + 5 * torch.randn((t, e), generator=g, device="cuda").clamp(-8, 8)
    z[::3] = -60 - 640 * torch.rand((len(z[::3]), e), generator=g, device="cuda")
    z[1::7, 0] = 1.5
    for bias in (None, torch.randn((e,), generator=g, device="cuda")):
        sel, w = _topk(z, u, bias=bias, scoring=scoring, scale=2.5)
        ids, want = ref.route(z.cpu().numpy(), u, None if bias is None else bias.cpu().numpy(), scoring, True, 2.5)
        assert np.array_equal(sel.cpu().numpy(), ids)
        np.testing.assert_allclose(w.cpu().numpy(), want, rtol=29 * 2.0 ** -24, atol=2.0 ** -126)
    if u == 1:
        assert (w == 2.5).all()


@pytest.mark.parametrize("e", [40, 300])
def test_equal_scores_below_the_range_of_fp32(e):
    z = torch.full((3, e), -150.0, device="cuda")
    z[2] = -800.0  # zero in 64 bits too
    for scoring in (1, 2):
        sel, w = _topk(z, 8, scoring=scoring)
        assert (sel == torch.arange(8, device="cuda")).all()
        assert (w[:2] == 0.125).all()
    assert (_topk(z, 8, scoring=1)[1][2] == 0).all()
    assert (_topk(z, 8, scoring=1, renormalize=False)[1] == 0).all()
