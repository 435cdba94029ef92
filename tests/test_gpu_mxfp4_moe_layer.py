"""GPU tests of mxfp4_moe_layer against the layer in 64 bits, with the tolerance
that mxfp4_ref.moe_layer derives; ids must be equal."""
import numpy as np
import pytest
import torch

from tests import mxfp4_ref as ref

pytestmark = pytest.mark.gpu


def _q8():
    import q8_quantized_matmul_amd as q8
    return q8


def _experts(rng, e, d, f):
    """Uniform codes with scales that keep gate and up around one."""
    lo = 127 - 5 - int(np.log2(d) / 2)
    return (ref.random_matrix(rng, (e, f, d), lo, lo + 1), ref.random_matrix(rng, (e, f, d), lo, lo + 1),
            ref.random_matrix(rng, (e, d, f), 118, 120))


def _run(x, logits, mats, n_used, out_dtype=torch.float32, **kw):
    q8 = _q8()
    return q8.mxfp4_moe_layer(x, logits, *(ref.device(q8, m) for m in mats), n_used, out_dtype=out_dtype, **kw)


def _check(x, logits, mats, n_used, out_dtype=torch.float32, tight=True, **kw):
    out, sel, w = _run(x, logits, mats, n_used, out_dtype, **kw)
    half = float(torch.finfo(out_dtype).eps) / 2
    opts = dict(kw)
    opts.pop("workspace", None)
    if opts.get("bias") is not None:
        opts["bias"] = opts["bias"].cpu().numpy()
    want, tol, ids, weights = ref.moe_layer(ref.host(x), logits.cpu().numpy(), *mats, n_used, half=half, **opts)
    assert np.array_equal(sel.cpu().numpy(), ids)
    # Below the smallest normal number the output's steps stop shrinking: half of
    # one is tiny * eps / 2 (fp16: values under 2^-14 lie 2^-24 apart).
    tol = tol + float(torch.finfo(out_dtype).tiny) * half
    err = np.abs(ref.host(out) - want)
    assert (err <= tol).all(), (int((~(err <= tol)).sum()), float(np.nanmax(err / tol)), int(np.isnan(err).sum()))
    # The tolerance itself must be tight: a wrong product would not fit in it.
    assert np.median(tol if tight else err) < 0.05 * np.abs(want).max() + half
    return out, sel, w


def _inputs(rng, t, d, e, dtype=torch.bfloat16):
    x = torch.from_numpy(rng.standard_normal((t, d)).astype(np.float32)).to(dtype).cuda()
    return x, torch.from_numpy(rng.standard_normal((t, e)).astype(np.float32) * 1.5).cuda()


SHAPES = [
    # t, d, f, e, u: one of everything; widths of one block, with K tails, of several steps
    (1, 32, 32, 1, 1), (1, 256, 128, 8, 2), (2, 96, 64, 5, 5), (5, 544, 96, 7, 3), (11, 1056, 352, 20, 4),
    (1, 4096, 256, 9, 8), (3, 512, 2080, 4, 2), (7, 736, 1024, 300, 6),
    # many tokens on few experts: several token tiles of one expert
    (16, 128, 128, 2, 1), (17, 128, 128, 2, 2), (33, 160, 64, 3, 2), (64, 96, 96, 2, 1), (64, 512, 128, 1, 1),
    (40, 288, 160, 512, 8), (64, 256, 64, 64, 32),
]


@pytest.mark.parametrize("t,d,f,e,u", SHAPES)
def test_shapes(t, d, f, e, u):
    rng = np.random.default_rng([t, d, f, e, u])
    x, z = _inputs(rng, t, d, e)
    _check(x, z, _experts(rng, e, d, f), u)


@pytest.mark.parametrize("t,d", [(2, 1024), (4, 1024), (6, 1024), (8, 1024), (9, 1024), (8, 8192), (8, 9216), (1, 65536), (1, 73728)])
def test_either_side_of_the_kernels_limits(t, d):
    """Token counts and widths on both sides of where x is quantized by every
    workgroup for itself, and the same token alone or among others."""
    rng = np.random.default_rng([t, d])
    x, z = _inputs(rng, t, d, 6)
    mats = _experts(rng, 6, d, 64)
    # A sum of d terms in fp32 may be off by d 2^-24 of the sum of their magnitudes,
    # which is sqrt(d) times the result: at 2^16 terms 2^-8 * 2^8, the result itself.
    # There the errors, and not their bound, are held against the results.
    tight = d < 2 ** 16
    _, sel, w = _check(x, z, mats, 3, tight=tight)
    one = _check(x[:1], z[:1], mats, 3, tight=tight)
    assert torch.equal(one[1], sel[:1]) and torch.equal(one[2], w[:1])


@pytest.mark.parametrize("x_dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_types(x_dtype, out_dtype):
    rng = np.random.default_rng(4)
    x, z = _inputs(rng, 9, 320, 12, x_dtype)
    _check(x, z, _experts(rng, 12, 320, 192), 3, out_dtype)


@pytest.mark.parametrize("scoring", [0, 1, 2])
@pytest.mark.parametrize("renormalize", [True, False])
def test_routing_options_and_clamp(scoring, renormalize):
    rng = np.random.default_rng(6)
    x, z = _inputs(rng, 13, 256, 10)
    b = torch.from_numpy(rng.standard_normal(10).astype(np.float32) * 0.3).cuda()
    mats = _experts(rng, 10, 256, 128)
    loud = (mats[0], (mats[1][0], mats[1][1] + 5), mats[2])  # up is large: the limits act
    a, _, _ = _check(x, z, loud, 4, bias=b, scoring=scoring, renormalize=renormalize, scale=1.5, clamp=10.0)
    c, _, _ = _check(x, z, loud, 4, bias=b, scoring=scoring, renormalize=renormalize, scale=1.5)
    assert not torch.equal(a, c)


def test_masked_experts_and_padded_rows():
    """Padding rows (all logits -inf) give zeros and ids of -1, also when the
    whole batch is padding; experts switched off everywhere are not read."""
    rng = np.random.default_rng(8)
    x, z = _inputs(rng, 20, 256, 12)
    mats = _experts(rng, 12, 256, 96)
    z[17:] = -float("inf")
    z[:, 3] = -float("inf")
    z[2, 2:] = -float("inf")     # two experts left for four slots
    for m in mats:
        m[1][3] = 255            # the switched-off expert is all NaN
    out, sel, w = _check(x, z, [(m[0], np.where(m[1] == 255, 127, m[1])) for m in mats], 4)
    nan_out, nan_sel, _ = _run(x, z, mats, 4)
    assert torch.equal(nan_out, out) and torch.equal(nan_sel, sel)
    assert (out[17:] == 0).all() and (sel[17:] == -1).all() and (w[17:] == 0).all()
    z[:] = -float("inf")
    out, sel, w = _run(x, z, mats, 4)
    assert (out == 0).all() and (sel == -1).all() and (w == 0).all()


def test_nan_stays_with_its_token_and_expert():
    rng = np.random.default_rng(9)
    x, z = _inputs(rng, 6, 256, 5, torch.float32)
    mats = _experts(rng, 5, 256, 64)
    base, sel, _ = _run(x, z, mats, 2)
    x2 = x.clone()
    x2[3, 100] = float("nan")
    out, _, _ = _run(x2, z, mats, 2)
    assert torch.isnan(out[3]).all() and torch.equal(out[[0, 1, 2, 4, 5]], base[[0, 1, 2, 4, 5]])
    z2 = z.clone()
    z2[1, 4] = float("nan")      # a NaN logit makes the token's weights NaN
    out, sel2, w = _run(x, z2, mats, 2)
    assert sel2[1, 0] == 4 and torch.isnan(w[1]).all() and torch.isnan(out[1]).all()
    assert torch.equal(out[[0, 2, 3, 4, 5]], base[[0, 2, 3, 4, 5]])
    mats[2][1][2, 7, 0] = 255    # one NaN block of expert 2's down: row 7 of its tokens
    out, _, _ = _run(x, z, mats, 2)
    hit = (sel == 2).any(1)
    assert hit.any() and torch.isnan(out[hit, 7]).all()
    out[:, 7] = base[:, 7]
    assert torch.equal(out, base)


def test_equals_its_parts():
    """The layer against the separate calls (quantize, products, quantize,
    products) of one token: gate, up and down are the same arithmetic up to
    summation order, which the 64-bit tolerance covers."""
    q8 = _q8()
    rng = np.random.default_rng(10)
    d, f, e, u = 512, 256, 6, 2
    x, z = _inputs(rng, 4, d, e)
    mats = _experts(rng, e, d, f)
    out, sel, w = _check(x, z, mats, u)
    dev = [ref.device(q8, m) for m in mats]
    part = lambda m, i: q8.Mxfp4(m.codes[i], m.scales[i])
    x4 = q8.mxfp4_quantize(x)
    want, tol, _, _ = ref.moe_layer(ref.host(x), z.cpu().numpy(), *mats, u)
    sel_r, w_r = q8.moe_topk(z, u)
    assert torch.equal(sel, sel_r) and torch.equal(w, w_r)
    for t in range(4):
        acc = torch.zeros(d, dtype=torch.float64, device="cuda")
        row = q8.Mxfp4(x4.codes[t:t + 1], x4.scales[t:t + 1])
        for j in range(u):
            i = int(sel[t, j])
            g, v = (q8.mxfp4_matmul(part(m, i), row) for m in dev[:2])
            mid = q8.mxfp4_quantize(torch.nn.functional.silu(g) * v)
            acc += w[t, j].double() * q8.mxfp4_matmul(part(dev[2], i), mid)[0].double()
        assert (np.abs(acc.cpu().numpy() - want[t]) <= tol[t]).all()
        assert (np.abs(ref.host(out[t]) - want[t]) <= tol[t]).all()


def test_order_of_tokens_does_not_matter():
    """A token's output does not depend on its neighbours beyond the order of
    fp32 sums: permuted batches give permuted outputs within tolerance, and a
    repeated call the same bits."""
    rng = np.random.default_rng(12)
    x, z = _inputs(rng, 30, 256, 9)
    mats = _experts(rng, 9, 256, 128)
    out, sel, w = _check(x, z, mats, 3)
    p = torch.randperm(30).cuda()
    out2, sel2, _ = _check(x[p].contiguous(), z[p].contiguous(), mats, 3)
    assert torch.equal(sel[p], sel2)
    out3, _, _ = _run(x, z, mats, 3)
    assert torch.equal(out, out3)


def test_unaligned_scales():
    q8 = _q8()
    rng = np.random.default_rng(13)
    x, z = _inputs(rng, 5, 256, 4)
    mats = _experts(rng, 4, 256, 128)

    def shifted(m):
        m = ref.device(q8, m)
        buf = torch.empty(m.scales.numel() + 1, dtype=torch.uint8, device="cuda")
        s = buf[1:].view(m.scales.shape)
        s.copy_(m.scales)
        return q8.Mxfp4(m.codes, s)
    a = q8.mxfp4_moe_layer(x, z, *(shifted(m) for m in mats), 2, out_dtype=torch.float32)
    b = _run(x, z, mats, 2)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("t,d,f,e,u", [(1, 1024, 256, 16, 4), (37, 256, 128, 12, 3)])
def test_graph_replays_and_shared_workspace(t, d, f, e, u):
    """Two captured layers on one scratch, replayed with new inputs and eager
    work between: every replay equals the eager call."""
    q8 = _q8()
    rng = np.random.default_rng(t)
    ws = q8.mxfp4_moe_layer_workspace(t, u, e, d, f)
    layers = []
    for _ in range(2):
        x, z = _inputs(rng, t, d, e)
        mats = [ref.device(q8, m) for m in _experts(rng, e, d, f)]
        layers.append((x, z, mats, [torch.empty((t, d), dtype=torch.bfloat16, device="cuda"),
                                    torch.empty((t, u), dtype=torch.int32, device="cuda"),
                                    torch.empty((t, u), device="cuda")]))
    call = lambda x, z, mats, o: q8.mxfp4_moe_layer(x, z, *mats, u, out=o[0], selected=o[1], weights=o[2], workspace=ws)
    for layer in layers:
        call(*layer)
    torch.cuda.synchronize()
    s, graphs = torch.cuda.Stream(), []
    with torch.cuda.stream(s):
        for layer in layers:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                call(*layer)
            graphs.append(g)
    for rep in range(3):
        for x, z, _, o in layers:
            x.copy_(torch.randn_like(x))
            z.copy_(torch.randn_like(z))
            o[0].fill_(float("nan"))
        ws.fill_(0x7B)
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for x, z, mats, o in layers:
            want = q8.mxfp4_moe_layer(x, z, *mats, u)
            assert all(torch.equal(a, b) for a, b in zip(o, want)), rep


def test_two_streams_with_their_own_workspaces():
    q8 = _q8()
    rng = np.random.default_rng(21)
    jobs = []
    for _ in range(2):
        x, z = _inputs(rng, 8, 512, 16)
        mats = [ref.device(q8, m) for m in _experts(rng, 16, 512, 256)]
        jobs.append((x, z, mats, q8.mxfp4_moe_layer_workspace(8, 4, 16, 512, 256), torch.cuda.Stream()))
    want = [q8.mxfp4_moe_layer(x, z, *m, 4)[0] for x, z, m, _, _ in jobs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (x, z, m, ws, s) in enumerate(jobs):
            with torch.cuda.stream(s):
                got[i].append(q8.mxfp4_moe_layer(x, z, *m, 4, workspace=ws)[0])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_full_size_sampled():
    """256 experts of 4096 x 2048, 64 tokens: the quantized weights of a
    normal draw; every expert's output of a few tokens against 64 bits."""
    q8 = _q8()
    t, d, f, e, u = 64, 4096, 2048, 256, 8
    g = torch.Generator(device="cuda").manual_seed(2)

    def experts(n, k):
        codes = torch.empty((e, n, k // 2), dtype=torch.uint8, device="cuda")
        scales = torch.empty((e, n, k // 32), dtype=torch.uint8, device="cuda")
        for i in range(e):
            q8.mxfp4_quantize(torch.randn((n, k), generator=g, device="cuda") * 0.02, codes=codes[i], scales=scales[i])
        return q8.Mxfp4(codes, scales)
    mats = [experts(f, d), experts(f, d), experts(d, f)]
    x = torch.randn((t, d), generator=g, device="cuda", dtype=torch.bfloat16)
    z = torch.randn((t, e), generator=g, device="cuda")
    out, sel, w = q8.mxfp4_moe_layer(x, z, *mats, u, out_dtype=torch.float32)
    ids, _ = ref.route(z.cpu().numpy(), u)
    assert np.array_equal(sel.cpu().numpy(), ids)
    for tok in (0, 41):
        use = sel[tok].sort().values.long()
        host = [(m.codes[use].cpu().numpy(), m.scales[use].cpu().numpy()) for m in mats]
        zt = z[tok:tok + 1, use].cpu().numpy()
        want, tol, _, _ = ref.moe_layer(ref.host(x[tok:tok + 1]), zt, *host, u)
        assert (np.abs(ref.host(out[tok:tok + 1]) - want) <= tol).all(), tok
    one, _, _ = q8.mxfp4_moe_layer(x[:1].contiguous(), z[:1].contiguous(), *mats, u, out_dtype=torch.float32)
    use = sel[0].sort().values.long()
    host = [(m.codes[use].cpu().numpy(), m.scales[use].cpu().numpy()) for m in mats]
    want, tol, _, _ = ref.moe_layer(ref.host(x[:1]), z[:1, use].cpu().numpy(), *host, u)
    assert (np.abs(ref.host(one) - want) <= tol).all()
