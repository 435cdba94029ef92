"""GPU tests of moe_topk, the MoE router, against a 64-bit form of the same
definition: equal ids, and weights within the roundings of fp32.

Weights: a softmax weight carries the rounding of z - m (half a step of a number
up to the logits' spread), of expf (one step), of a sum of at most 1024
positive terms (16 register additions and 6 across lanes, or fewer) and of
three more operations; the other scores start as one rounding of a 64-bit value.
"""
import numpy as np
import pytest
import torch

from tests import mxfp4_ref as ref

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -24  # half a step of fp32, relative


def _q8():
    import q8_quantized_matmul_amd as q8
    return q8


def _check(logits, n_used, bias=None, scoring=0, renormalize=True, scale=1.0):
    q8 = _q8()
    sel, w = q8.moe_topk(logits, n_used, bias=bias, scoring=scoring, renormalize=renormalize, scale=scale)
    z = logits.cpu().numpy()
    ids, want = ref.route(z, n_used, None if bias is None else bias.cpu().numpy(), scoring, renormalize, scale)
    assert np.array_equal(sel.cpu().numpy(), ids)
    fin = z[np.isfinite(z) & (z > -1e30)]  # the rest: exp is 0, or z - m is
    spread = float(fin.max() - fin.min()) if fin.size else 0.0
    tol = (spread + 2 + 24 + 4) * HALF if scoring == 0 else (1 + 24 + 4) * HALF
    np.testing.assert_allclose(w.cpu().numpy(), want, rtol=tol, atol=2.0 ** -126)
    return sel, w


@pytest.mark.parametrize("scoring", [0, 1, 2])
@pytest.mark.parametrize("t,e,u", [(1, 1, 1), (1, 256, 8), (5, 7, 7), (3, 64, 32), (67, 65, 6), (9, 200, 8), (130, 500, 4), (4, 1024, 32)])
def test_shapes(t, e, u, scoring):
    g = torch.Generator(device="cuda").manual_seed(t * e + u)
    z = torch.randn((t, e), generator=g, device="cuda") * 2
    b = torch.randn((e,), generator=g, device="cuda") * 0.2
    for renorm in (True, False):
        _check(z, u, None, scoring, renorm)
        _check(z, u, b, scoring, renorm, 2.5)


@pytest.mark.parametrize("scoring", [0, 1, 2])
def test_ties_take_the_lowest_ids(scoring):
    z = torch.randint(-2, 3, (40, 150), device="cuda").float()
    z[0] = 1.25
    sel, _ = _check(z, 8, None, scoring)
    assert sel[0].tolist() == list(range(8))
    z[1] = 0.0
    z[1, ::2] = -0.0  # equal numbers: the sign of a zero does not order
    for b in (None, torch.zeros(150, device="cuda"), torch.full((150,), -0.0, device="cuda")):
        sel = _q8().moe_topk(z[1:2].contiguous(), 4, bias=b, scoring=scoring)[0]
        assert sel[0].tolist() == [0, 1, 2, 3]


@pytest.mark.parametrize("scoring", [0, 1, 2])
def test_masked_experts_and_empty_rows(scoring):
    z = torch.randn((12, 40), device="cuda")
    z[0] = -float("inf")
    z[1, 3:] = -float("inf")      # three experts left for eight slots
    z[2, :39] = -float("inf")
    z[3] = torch.finfo(torch.float32).min
    z[4, ::2] = torch.finfo(torch.float32).min
    b = torch.zeros(40, device="cuda")
    b[5] = -float("inf")          # switched off by the bias
    sel, w = _check(z, 8, None, scoring)
    assert (sel[0] == -1).all() and (w[0] == 0).all()
    assert (sel[1, 3:] == -1).all() and (w[1, 3:] == 0).all()
    sel, _ = _check(z, 8, b, scoring)
    assert not (sel == 5).any()
    _check(z, 8, None, scoring, renormalize=False)


@pytest.mark.parametrize("e,u", [(40, 8), (130, 8), (256, 32), (500, 5), (1024, 32)])
@pytest.mark.parametrize("scoring", [0, 1, 2])
def test_nearly_equal_scores(scoring, e, u):
    """Logits a few steps of fp32 apart, logits whose sigmoid is 1, small scores far
    apart as numbers but not as fp32 sums, and a bias that makes them all one."""
    g = torch.Generator(device="cuda").manual_seed(e + u + scoring)
    step = torch.randint(0, 40, (6, e), generator=g, device="cuda").float()
    z = 1 + step * 2.0 ** -23
    z[1] = 38 + step[1]
    z[2] = -70 - step[2] / 4
    z[3] = -70 - torch.rand((e,), generator=g, device="cuda") * 10
    z[4] = -step[4] * 2.0 ** -140  # subnormal
    z[5, e // 3:] = -float("inf")
    _check(z, u, None, scoring)
    _check(z, u, torch.full((e,), 3.0, device="cuda"), scoring)
    b = torch.randn((e,), generator=g, device="cuda")
    b[1::3] = 1e30
    b[2::7] = -1e30
    _check(z, u, b, scoring)


def test_infinite_and_nan_biases():
    z = torch.randn((5, 300), device="cuda")
    b = torch.zeros(300, device="cuda")
    b[7] = b[290] = float("inf")
    b[11] = float("nan")
    b[20:200] = -float("inf")
    for scoring in (0, 1, 2):
        sel, _ = _q8().moe_topk(z, 6, bias=b, scoring=scoring)
        ids, _ = ref.route(z.cpu().numpy(), 6, b.cpu().numpy(), scoring)
        assert np.array_equal(sel.cpu().numpy(), ids)
        assert (sel[:, :3] == torch.tensor([11, 7, 290], device="cuda")).all()


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("scoring", [0, 1, 2])
def test_nan_and_infinite_logits(scoring, renormalize):
    q8 = _q8()
    z = torch.randn((3, 70), device="cuda")
    z[0, 66] = float("nan")
    z[1, 9] = float("inf")
    sel, w = q8.moe_topk(z, 4, scoring=scoring, renormalize=renormalize)
    ids, want = ref.route(z.cpu().numpy(), 4, None, scoring, renormalize)
    assert np.array_equal(sel.cpu().numpy(), ids)
    assert np.array_equal(np.isnan(w.cpu().numpy()), np.isnan(want))
    assert sel[0, 0] == 66 and sel[1, 0] == 9 and torch.isfinite(w[2]).all()


def test_softmax_over_chosen_far_below_the_largest_logit():
    """A bias may choose experts whose logits lie far below others: the softmax
    over the chosen does not underflow."""
    z = torch.zeros((2, 16), device="cuda")
    z[:, 0] = 500.0
    b = torch.zeros(16, device="cuda")
    b[0] = -1000.0
    _, w = _check(z, 4, b, 0)
    assert torch.equal(w, torch.full((2, 4), 0.25, device="cuda"))


def test_feeds_the_q8_expert_calls():
    """selected / weights drive q8_0_moe_ffn: the same output as from lists made
    on the host."""
    q8 = _q8()
    d, f, e, t, u = 256, 128, 6, 5, 3
    g = torch.Generator(device="cuda").manual_seed(5)
    mk = lambda r, c: torch.stack([q8.q8_0_quantize_act(torch.randn((r, c), generator=g, device="cuda") * 0.05) for _ in range(e)])
    gate, up, down = mk(f, d), mk(f, d), mk(d, f)
    x = q8.q8_0_quantize_act(torch.randn((t, d), generator=g, device="cuda"))
    z = torch.randn((t, e), generator=g, device="cuda")
    sel, w = q8.moe_topk(z, u)
    tables = [q8.expert_table(m) for m in (gate, up, down)]
    out, _ = q8.q8_0_moe_ffn(*tables, e, sel, w, x, d, f)
    ids, _ = ref.route(z.cpu().numpy(), u)
    out2, _ = q8.q8_0_moe_ffn(*tables, e, torch.from_numpy(ids).cuda(), w, x, d, f)
    assert torch.isfinite(out).all() and torch.equal(out, out2)


def test_graph_replays():
    q8 = _q8()
    z = torch.randn((33, 256), device="cuda")
    sel = torch.empty((33, 8), dtype=torch.int32, device="cuda")
    w = torch.empty((33, 8), device="cuda")
    q8.moe_topk(z, 8, selected=sel, weights=w)
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        q8.moe_topk(z, 8, selected=sel, weights=w)
    for rep in range(3):
        z.copy_(torch.randn((33, 256), device="cuda"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        a, b = q8.moe_topk(z, 8)
        assert torch.equal(sel, a) and torch.equal(w, b), rep
