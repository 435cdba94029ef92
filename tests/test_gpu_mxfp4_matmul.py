"""GPU tests of mxfp4_matmul against the product in 64 bits.

Tolerance: products are exact and the fp32 sum of k terms is made of at most
k / 32 + 8 roundings (one an instruction of 64 or 128 values with its own
alignment, and the joins of splits), each at most a step of fp32 of the
partial sum, which sum |w x| bounds; then half a step of the output type."""
import numpy as np
import pytest
import torch

from tests import mxfp4_ref as ref

pytestmark = pytest.mark.gpu


def _q8():
    import q8_quantized_matmul_amd as q8
    return q8


def _bound(w, x, want, dtype):
    k = w.shape[1]
    mag = np.abs(x) @ np.abs(w).T
    half = float(torch.finfo(dtype).eps) / 2
    # Half a step of the output: relative, and of its subnormals (fp16 numbers
    # under 2^-14 lie 2^-24 apart); fp32 rounds nothing, but may flush below 2^-126.
    out = half * np.abs(want) + float(torch.finfo(dtype).tiny) * half if dtype != torch.float32 else 2.0 ** -126
    return (k / 32 + 8) * 2.0 ** -23 * mag + out


def _check(out, w, x, rows=None):
    """out [t][n] against the product of the float64 matrices; rows: tokens to check."""
    rows = slice(None) if rows is None else rows
    want = x[rows] @ w.T
    got = ref.host(out)[rows]
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    err, tol = np.abs(got - want), _bound(w, x[rows], want, out.dtype)
    bad = ~nan & ~(err <= tol)
    assert not bad.any(), (bad.sum(), np.nanmax(err / tol))


def _case(k, n, t, seed=0, **kw):
    rng = np.random.default_rng([k, n, t, seed])
    return ref.random_matrix(rng, (n, k), **kw), ref.random_matrix(rng, (t, k), **kw)


SHAPES = [
    # k, n, t: one block; rows and tokens that fill no tile; K tails of 1..3 blocks
    (32, 1, 1), (32, 17, 3), (64, 16, 16), (96, 33, 5), (160, 100, 31), (544, 67, 9),
    # steps of 512: exactly one, one and a block, several
    (512, 48, 1), (544, 48, 2), (1024, 520, 1), (4096, 512, 1), (4096, 130, 12), (2912, 1000, 13),
    # token tiles and their edges
    (256, 64, 15), (256, 64, 17), (1056, 96, 32), (1056, 96, 33), (512, 200, 48), (512, 200, 63), (512, 200, 64),
    # above 64 tokens, ragged everywhere
    (256, 128, 65), (288, 129, 127), (1024, 257, 128), (1056, 300, 130), (2080, 260, 257), (4096, 100, 200),
    (512, 1000, 513), (32, 300, 300), (8192, 64, 100),
    # long K
    (32768, 40, 1), (32768, 64, 20), (16384, 256, 256),
]


@pytest.mark.parametrize("k,n,t", SHAPES)
def test_shapes(k, n, t):
    q8 = _q8()
    w, x = _case(k, n, t)
    out = q8.mxfp4_matmul(ref.device(q8, w), ref.device(q8, x))
    _check(out, ref.values(*w), ref.values(*x))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("k,n,t", [(96, 33, 5), (1024, 514, 1), (512, 130, 40), (1024, 260, 300)])
def test_output_types(k, n, t, dtype):
    q8 = _q8()
    w, x = _case(k, n, t, lo=120, hi=124)
    out = q8.mxfp4_matmul(ref.device(q8, w), ref.device(q8, x), out_dtype=dtype)
    assert out.dtype == dtype
    _check(out, ref.values(*w), ref.values(*x))


@pytest.mark.parametrize("k,n,t", [(1024, 64, 3), (1024, 64, 40), (1024, 256, 300)])
def test_extreme_scales_and_nan_blocks(k, n, t):
    """Scale bytes over the whole range with products that stay normal, and
    NaN blocks on both sides: only their rows and tokens are NaN."""
    q8 = _q8()
    rng = np.random.default_rng([k, n, t])
    w = ref.random_matrix(rng, (n, k), 0, 60)
    x = ref.random_matrix(rng, (t, k), 194, 254)
    w[1][n // 2, 3] = 255
    x[1][t - 1, k // 32 - 1] = 255
    out = q8.mxfp4_matmul(ref.device(q8, w), ref.device(q8, x))
    _check(out, ref.values(*w), ref.values(*x))


@pytest.mark.parametrize("k,n,t", [(1024, 64, 3), (1024, 300, 200)])
def test_unaligned_scales_and_row_slices(k, n, t):
    """Scale arrays at any byte, and rows cut out of a larger matrix; the rows
    around the output stay as they were."""
    q8 = _q8()
    w, x = _case(k, n, t)
    dw, dx = ref.device(q8, w), ref.device(q8, x)

    def shifted(m):
        buf = torch.empty(m.scales.numel() + 3, dtype=torch.uint8, device="cuda")
        s = buf[3:].view(m.scales.shape)
        s.copy_(m.scales)
        return q8.Mxfp4(m.codes, s)
    base = q8.mxfp4_matmul(dw, dx)
    assert torch.equal(q8.mxfp4_matmul(shifted(dw), shifted(dx)), base) or t > 64
    _check(q8.mxfp4_matmul(shifted(dw), shifted(dx)), ref.values(*w), ref.values(*x))
    out = torch.full((t + 2, n - 7), 3.0, device="cuda")
    q8.mxfp4_matmul(q8.Mxfp4(dw.codes[5:n - 2], dw.scales[5:n - 2]), dx, out=out[1:-1])
    _check(out[1:-1], ref.values(*w)[5:n - 2], ref.values(*x))
    assert (out[0] == 3.0).all() and (out[-1] == 3.0).all()


@pytest.mark.parametrize("k,n,t", [(4096, 2048, 200), (32768, 1024, 300), (1024, 32768, 1), (4096, 4096, 1024), (32768, 1024, 1)])
def test_large_shapes_sampled(k, n, t):
    q8 = _q8()
    w, x = _case(k, n, t)
    dw, dx = ref.device(q8, w), ref.device(q8, x)
    out = q8.mxfp4_matmul(dw, dx, out_dtype=torch.float32)
    rows = sorted({0, t // 3, t // 2, t - 1})
    _check(out, ref.values(*w), ref.values(*x), rows)
    assert torch.equal(out, q8.mxfp4_matmul(dw, dx)), "a second call differs"


def test_without_workspace():
    """Every plan falls back to one that needs no scratch; results within tolerance."""
    q8 = _q8()
    for k, n, t in ((32768, 64, 1), (16384, 256, 256), (32768, 130, 40)):
        w, x = _case(k, n, t)
        dw, dx = ref.device(q8, w), ref.device(q8, x)
        none = torch.empty(0, dtype=torch.uint8, device="cuda")
        _check(q8.mxfp4_matmul(dw, dx, workspace=none), ref.values(*w), ref.values(*x))
        half = torch.empty(q8.mxfp4_matmul_workspace_bytes(k, n, t) // 2, dtype=torch.uint8, device="cuda")
        _check(q8.mxfp4_matmul(dw, dx, workspace=half), ref.values(*w), ref.values(*x))


@pytest.mark.parametrize("k,n,t", [(32768, 1024, 1), (1024, 96, 20), (16384, 256, 256)])
def test_graph_replays_and_shared_workspace(k, n, t):
    """Two captured calls that share a scratch, replayed with eager work between:
    every replay equals the eager result."""
    q8 = _q8()
    cases = [_case(k, n, t, seed) for seed in (1, 2)]
    dev = [(ref.device(q8, w), ref.device(q8, x)) for w, x in cases]
    ws = q8.mxfp4_matmul_workspace(k, n, t)
    eager = [q8.mxfp4_matmul(w, x, workspace=ws).clone() for w, x in dev]
    outs = [torch.empty_like(e) for e in eager]
    torch.cuda.synchronize()
    s, graphs = torch.cuda.Stream(), []
    with torch.cuda.stream(s):
        for (w, x), o in zip(dev, outs):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                q8.mxfp4_matmul(w, x, out=o, workspace=ws)
            graphs.append(g)
    for rep in range(3):
        for o in outs:
            o.fill_(float("nan"))
        ws.fill_(0xC3)
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, e in zip(outs, eager):
            assert torch.equal(o, e), rep


def test_quantize_then_multiply():
    """The chain a program runs: quantize weights and activations, multiply."""
    q8 = _q8()
    wf = torch.randn((200, 736), device="cuda", dtype=torch.bfloat16)
    xf = torch.randn((21, 736), device="cuda", dtype=torch.float16)
    w, x = q8.mxfp4_quantize(wf), q8.mxfp4_quantize(xf)
    out = q8.mxfp4_matmul(w, x)
    _check(out, ref.values(*ref.quantize(ref.host(wf))), ref.values(*ref.quantize(ref.host(xf))))


# Lengths that every tile shape splits into an even count of stages, into one that is
# not a multiple of four, and unevenly; each regime's neighbours.
@pytest.mark.parametrize("k,n,t", [
    (17984, 1024, 4096), (17408, 7168, 512), (17696, 2048, 2048), (20000, 1000, 2500),
    (9216, 512, 512), (5184, 640, 200), (7168, 2048, 129), (11296, 300, 700), (4128, 1024, 64), (33056, 96, 100),
    (16416, 128, 33), (24640, 1024, 9), (40992, 256, 1), (2048, 8192, 32), (544, 64, 17), (512, 4096, 257),
])
def test_every_split_sums_every_value_once(k, n, t):
    """Codes at scale 1 make products that are multiples of 1/4 and sums below 2^22:
    every order of summation in fp32 is exact, and the result equals the 64-bit one."""
    q8 = _q8()
    g = torch.Generator(device="cuda").manual_seed(k + n + t)
    w, x = (q8.Mxfp4(torch.randint(0, 256, (r, k // 2), dtype=torch.uint8, device="cuda", generator=g),
                     torch.full((r, k // 32), 127, dtype=torch.uint8, device="cuda")) for r in (n, t))
    assert k * 36 * 4 < 2 ** 24
    want = q8.mxfp4_dequantize(x).double() @ q8.mxfp4_dequantize(w).double().t().contiguous()
    assert torch.equal(q8.mxfp4_matmul(w, x).double(), want)


@pytest.mark.parametrize("k,n,t", [(17984, 1024, 4096), (17408, 7168, 512), (8736, 512, 300), (40992, 256, 1), (5184, 640, 200)])
def test_a_larger_workspace_changes_nothing(k, n, t):
    q8 = _q8()
    g = torch.Generator(device="cuda").manual_seed(k)
    w, x = (q8.Mxfp4(torch.randint(0, 256, (r, k // 2), dtype=torch.uint8, device="cuda", generator=g),
                     torch.randint(118, 122, (r, k // 32), dtype=torch.uint8, device="cuda", generator=g)) for r in (n, t))
    need = q8.mxfp4_matmul_workspace_bytes(k, n, t)
    more = torch.empty(4 * need + 256, dtype=torch.uint8, device="cuda")
    assert torch.equal(q8.mxfp4_matmul(w, x), q8.mxfp4_matmul(w, x, workspace=more))
