"""kv8_attention against its plain 64-bit form, at the sizes and masks where it can go
wrong, and the cache's operators together as a step makes them."""
import numpy as np
import pytest
import torch

from tests.helpers import say
from tests.kv8_helpers import DTYPES, Case

pytestmark = pytest.mark.gpu

SIZES = {
    "one": [(1, 1)],
    "decode": [(1, 1), (1, 2), (1, 33), (1, 400), (1, 0), (1, 64)],
    "drafts": [(3, 40), (1, 1), (0, 12), (4, 4), (2, 300), (4, 2), (1, 0)],
    "prompt": [(37, 37), (70, 129), (1, 90), (0, 0), (130, 150)],
}


def run(c, q, kernel=0, **kw):
    lse = torch.full((c.n_tok, q.shape[1]), 5.0, device="cuda")
    batch = kw.pop("batch", c.batch)
    if kernel:
        out = c.q8.kv8_attention_debug(c.cache, batch, q, kernel, lse=lse, **kw)
    else:
        out = c.q8.kv8_attention(c.cache, batch, q, lse=lse, **kw)
    torch.cuda.synchronize()
    return out, lse


# the two kernels, whatever the sizes would choose
both = pytest.mark.parametrize("kernel", [1, 2])


@both
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("d,hq,hkv", [(64, 6, 3), (128, 4, 2), (192, 2, 2), (256, 8, 1), (512, 5, 1)])
@pytest.mark.parametrize("sizes", list(SIZES))
def test_attention(sizes, d, hq, hkv, dtype, kernel):
    say("attention", sizes, d, hq, hkv, dtype, kernel)
    if kernel == 2 and d == 512 and dtype == "fp32":
        pytest.skip("the tiled kernel has no such variant")
    c = Case(SIZES[sizes], hkv, d, seed=d + hq, stale=np.nan, one_row=sizes in ("one", "decode")).upload()
    q, q64 = c.rows(hq, DTYPES[dtype], spread=1.5)
    out, lse = run(c, q, kernel)
    assert out.dtype == q.dtype
    say("worst", c.check_attention(q, q64, out, lse))


@both
@pytest.mark.parametrize("group", [1, 3, 5, 16, 17, 32, 64])
def test_groups(group, kernel):
    c = Case([(1, 70), (2, 35), (1, 5)], 2, 64, seed=group).upload()
    q, q64 = c.rows(2 * group, torch.bfloat16)
    out, lse = run(c, q, kernel)
    c.check_attention(q, q64, out, lse)


@both
@pytest.mark.parametrize("page,block", [(16, 16), (32, 32), (256, 16), (128, 128), (1024, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_pages_and_blocks(page, block, dtype, kernel):
    c = Case([(1, 500), (90, 210), (1, 129), (17, 17)], 2, 64, page, block, seed=page, stale=np.inf).upload()
    q, q64 = c.rows(4, DTYPES[dtype])
    out, lse = run(c, q, kernel)
    c.check_attention(q, q64, out, lse)


@both
@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 64, 100, 1000])
@pytest.mark.parametrize("sizes", ["decode", "prompt"])
def test_windows(window, sizes, kernel):
    c = Case(SIZES[sizes], 2, 64, 16, seed=window, stale=np.nan).upload()
    # what no window reaches must not matter: NaN scales there
    for s, (n, m) in enumerate(c.sizes):
        last = m - n - window + 1  # first key of the first row
        for blk in range(max(last, 0) // 16):
            c.ks[c.table[s, blk], :, 0] = np.nan
            c.vs[c.table[s, blk], :, 0] = np.nan
    c.upload()
    q, q64 = c.rows(4, torch.float16)
    out, lse = run(c, q, kernel, window=window)
    c.check_attention(q, q64, out, lse, window=window)


@both
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("spread", [0.5, 20.0, 300.0])
def test_sinks(dtype, spread, kernel):
    """Sinks far below, among and far above the scores; rows without keys have only the sink."""
    c = Case(SIZES["drafts"] + [(40, 80)], 2, 64, seed=9).upload()
    q, q64 = c.rows(6, DTYPES[dtype])
    sinks = (torch.randn(6, generator=torch.Generator().manual_seed(1)) * spread).cuda()
    out, lse = run(c, q, kernel, sinks=sinks)
    c.check_attention(q, q64, out, lse, sinks=sinks)


@both
@pytest.mark.parametrize("q_type", list(DTYPES))
@pytest.mark.parametrize("out_type", list(DTYPES))
def test_output_types(q_type, out_type, kernel):
    c = Case([(1, 100), (50, 60)], 1, 128, seed=2).upload()
    q, q64 = c.rows(4, DTYPES[q_type])
    out, lse = run(c, q, kernel, out_dtype=DTYPES[out_type])
    assert out.dtype == DTYPES[out_type]
    c.check_attention(q, q64, out, lse)


@pytest.mark.parametrize("n_new", [1, 24, 80])
@pytest.mark.parametrize("splits", [0, 2, 7, 64])
def test_splits(n_new, splits):
    """Long sequences on fewer and more splits than the plan's, by the workspace that they get."""
    c = Case([(n_new, 3000 + n_new), (n_new, 17 + n_new), (0, 40)], 1, 64, page=256, seed=splits).upload()
    q, q64 = c.rows(4, torch.bfloat16)
    need = c.q8.kv8_attention_workspace_bytes(c.cache, c.batch, 4)
    ws = torch.full((min(need, splits * c.n_tok * 4 * 65 * 4),), 255, dtype=torch.uint8, device="cuda")
    out, lse = run(c, q, workspace=ws)
    c.check_attention(q, q64, out, lse)
    again, _ = run(c, q, workspace=ws)
    assert torch.equal(out, again)


@both
@pytest.mark.parametrize("splits", [2, 3, 11])
@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_forced_splits(d, splits, kernel):
    c = Case([(40, 700), (1, 90), (0, 10), (9, 33)], 1, d, seed=splits).upload()
    q, q64 = c.rows(3, torch.bfloat16)
    sinks = torch.tensor([0.5, -30.0, 4.0], device="cuda")
    out, lse = run(c, q, kernel, splits=splits, sinks=sinks)
    c.check_attention(q, q64, out, lse, sinks=sinks)
    assert torch.equal(out, run(c, q, kernel, splits=splits, sinks=sinks)[0])


@both
def test_long_prompts(kernel):
    """Many tiles, the workgroups' last ones partly filled, sequences that end inside a tile of rows."""
    c = Case([(300, 300), (517, 900), (65, 1000), (1, 3)], 1, 128, seed=21, stale=np.nan).upload()
    q, q64 = c.rows(3, torch.bfloat16)
    out, lse = run(c, q, kernel)
    c.check_attention(q, q64, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("sizes", [((1024, 1024), (700, 1500)), ((2500, 2500), (2500, 2500))])
def test_kernels_agree(sizes, dtype):
    """The library's choice is one of the two kernels, the tiled one (with some splits or none) for the longer
    prompts, and both give the same within their bounds."""
    c = Case(list(sizes), 8, 64, seed=22).upload()
    q, _ = c.rows(32, DTYPES[dtype])
    auto, lse = run(c, q)
    tiled, lse1 = run(c, q, 2)
    stream, lse2 = run(c, q, 1)
    assert not torch.equal(tiled, stream)
    assert (any(torch.equal(auto, run(c, q, 2, splits=n)[0]) for n in (1, 2, 3, 4))
            or (torch.equal(auto, stream) and sizes[0][0] < 2000))
    vmax = 127 / 60
    assert (tiled.float() - stream.float()).abs().max() <= 2 * vmax * (2.0 ** -11 + torch.finfo(DTYPES[dtype]).eps)
    assert (lse1 - lse2).abs().max() <= 2.0 ** -12


@both
def test_scores_of_any_size(kernel):
    """Scores in the thousands (one key takes all), equal scores, and a scale of zero."""
    c = Case([(1, 300), (20, 90)], 2, 64, seed=4).upload()
    q, q64 = c.rows(2, torch.float32, spread=300.0)
    for scale in (4.0, -4.0, 0.0, 1e-30):
        out, lse = run(c, q, kernel, scale=scale)
        c.check_attention(q, q64, out, lse, scale=scale)


@both
def test_scales_of_any_size(kernel):
    """Blocks whose scales lie far apart, zero and subnormal ones among them."""
    for lo, hi in ((-30, 30), (-140, -100), (-60, 0)):
        c = Case([(1, 400), (33, 70)], 2, 64, 16, seed=5)
        c.vs[:] = (2.0 ** c.rng.uniform(lo, hi, c.vs.shape)).astype(np.float32)
        c.vs[::3] = 0.0
        c.ks[::4] = 0.0
        c.upload()
        q, q64 = c.rows(2, torch.float32)
        out, lse = run(c, q, kernel)
        c.check_attention(q, q64, out, lse)


@both
def test_growing_scores(kernel):
    """Each key scores above all before it by more than the slack of the running bound."""
    c = Case([(1, 200), (60, 200)], 1, 64, 16, seed=6)
    c.k[:] = 0
    c.k[..., 0] = 100
    for s, (n, m) in enumerate(c.sizes):
        for blk in range(-(-m // 16)):
            c.ks[c.table[s, blk], 0, 0] = 0.01 * (blk + 1)
    c.upload()
    for spread in (3.0, 100.0):
        q, _ = c.rows(1, torch.float32)
        q = q.abs() * spread
        out, lse = run(c, q, kernel, scale=1.0)
        c.check_attention(q, q.double().cpu().numpy(), out, lse, scale=1.0)


@both
def test_queries_of_any_size(kernel):
    """Rows of very large and small queries, of zeros, and with a NaN or an infinity: that row alone is NaN."""
    c = Case([(1, 90), (40, 64)], 1, 64, seed=7).upload()
    q, _ = c.rows(2, torch.float32)
    q[3] *= 1e30
    q[4] *= 1e-30
    q[5] = 0
    q[6, 0] *= 1e-38
    q[8, 1, 4] = float("nan")
    q[9, 0, 63] = float("inf")
    out, lse = run(c, q, kernel, scale=1.0)
    got = out.cpu()
    bad = torch.zeros(c.n_tok, 2, dtype=torch.bool)
    bad[8, 1] = bad[9, 0] = True
    assert torch.equal(got.isnan().all(-1), bad) and torch.equal(got.isnan().any(-1), bad)
    clean = torch.where(bad[..., None].cuda(), torch.zeros_like(q), q)
    clean_out, clean_lse = run(c, clean, kernel, scale=1.0)
    assert torch.equal(torch.where(bad[..., None], 0, clean_out.cpu()), torch.where(bad[..., None], 0, got))
    clean[3] = 0  # scores of 1e30 times the others': the one-key limit, where the plain form's bound says nothing
    clean_out, clean_lse = run(c, clean, kernel, scale=1.0)
    c.check_attention(clean, clean.double().cpu().numpy(), clean_out, clean_lse, scale=1.0)


@both
def test_nan_blocks_reach_their_readers_only(kernel):
    c = Case([(1, 100), (90, 100), (3, 50)], 1, 64, 16, seed=8)
    c.ks[c.table[1, 3]] = np.nan   # tokens 48 .. 63
    c.vs[c.table[2, 2]] = np.nan   # tokens 32 .. 47
    c.upload()
    q, q64 = c.rows(3, torch.bfloat16)
    out, lse = run(c, q, kernel)
    c.check_attention(q, q64, out, lse if False else None)
    assert out[1:39].isfinite().all() and out[39:91].isnan().all() and out[0].isfinite().all()


@both
def test_bad_pages_give_nan(kernel):
    c = Case([(1, 300), (1, 300), (100, 300), (1, 40)], 1, 64, 64, seed=10)
    c.table[0, 2] = -1
    c.table[2, 3] = c.k.shape[0]  # tokens 192 .. 255: the rows behind see them
    c.upload()
    q, q64 = c.rows(2, torch.float32)
    out, lse = run(c, q, kernel)
    c.check_attention(q, q64, out)
    assert out[0].isnan().all() and out[1].isfinite().all() and out[2:102].isnan().all() and out[102].isfinite().all()


def test_rows_behind_the_last_sequence():
    c = Case([(1, 700), (30, 40)], 1, 64).upload()
    q = torch.randn(40, 2, 64, device="cuda")
    table, lens, starts = (torch.from_numpy(a).cuda() for a in (c.table, c.lens, c.starts))
    b = c.q8.Kv8Batch(table, lens, starts, n_tok=40, max_new=30)
    for ws in (None, torch.empty(0, dtype=torch.uint8, device="cuda")):
        out, lse = torch.full_like(q, 7.0), torch.full((40, 2), 7.0, device="cuda")
        c.q8.kv8_attention(c.cache, b, q, out=out, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        assert (out[31:] == 7).all() and (lse[31:] == 7).all() and not (out[:31] == 7).any()


@both
@pytest.mark.parametrize("offset", [0, 1, 8])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_strided_queries(offset, dtype, kernel):
    c = Case([(20, 77), (1, 4)], 2, 64).upload()
    x, x64 = c.rows(7, DTYPES[dtype])
    flat = torch.zeros(c.n_tok, 7 * 64 + 24, dtype=DTYPES[dtype], device="cuda")
    flat[:, offset:offset + 7 * 64] = x.view(c.n_tok, -1)
    q = flat[:, offset:offset + 7 * 64].unflatten(1, (7, 64))[:, 1:5]
    out, lse = run(c, q, kernel)
    c.check_attention(q, x64[:, 1:5], out, lse)
    by_head = x[:, 1:5].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(out, run(c, by_head, kernel)[0])
    same = x[:, :1].expand(-1, 4, -1)  # one query for all heads
    out, lse = run(c, same, kernel)
    c.check_attention(same, np.repeat(x64[:, :1], 4, 1), out, lse)


def test_large_pool_offsets():
    """Pages whose codes lie beyond 2^31 and 2^32 bytes."""
    import q8_quantized_matmul_amd as q8
    c = Case([(1, 200), (70, 150)], 1, 512, 1024, 128, seed=11).upload()
    per = 1024 * 512
    n = 2 ** 32 // per + 40
    k, v = (torch.zeros(n, 1, 1024, 512, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(n, 1, 8, device="cuda") for _ in range(2))
    far = {int(p): n - 1 - i for i, p in enumerate(c.table[:, 0])}
    table = torch.from_numpy(c.table).cuda()
    for i, p in enumerate(c.table[:, 0]):
        to = far[int(p)] if i else 2 ** 31 // per + 1
        k[to], v[to], ks[to], vs[to] = c.cache.k[p], c.cache.v[p], c.cache.k_scales[p], c.cache.v_scales[p]
        table[i, 0] = to
    big = q8.Kv8Cache(k, v, ks, vs)
    batch = q8.Kv8Batch(table, c.batch.lens, c.batch.starts, n_tok=c.n_tok)
    q, _ = c.rows(4, torch.bfloat16)
    assert torch.equal(q8.kv8_attention(big, batch, q), q8.kv8_attention(c.cache, c.batch, q))
    x, _ = c.rows(1, torch.bfloat16)
    q8.kv8_write(big, batch, x, x)
    q8.kv8_write(c.cache, c.batch, x, x)
    for a, b in zip(q8.kv8_read(big, batch), q8.kv8_read(c.cache, c.batch)):
        assert torch.equal(a, b)


def test_step_in_a_graph():
    """A decode step (write, attend) captured once and replayed while the sequences grow over
    block and page borders, eager work in between; two graphs share a workspace."""
    c = Case([(1, 30), (1, 63), (1, 1), (1, 500)], 2, 128, 64, one_row=True, seed=12)
    c.table = np.concatenate([c.table, np.full((4, 2), -5, np.int32)], 1)
    extra = c.k.shape[0]
    for name in ("k", "v", "ks", "vs"):
        a = getattr(c, name)
        setattr(c, name, np.concatenate([a, a[:4]]))
    for s, m in enumerate(c.lens):  # the page that each grows into
        c.table[s, -(-int(m) // 64)] = extra + s
    c.upload()
    q8 = c.q8
    lens = torch.from_numpy(c.lens.copy()).cuda()
    batch = q8.Kv8Batch(torch.from_numpy(c.table).cuda(), lens, max_len=600)
    q, k, v = (torch.zeros(4, h, 128, dtype=torch.bfloat16, device="cuda") for h in (8, 2, 2))
    out, out2 = torch.empty_like(q), torch.empty_like(q)
    ws = q8.kv8_attention_workspace(c.cache, batch, 8)
    assert ws.numel() > 0
    graphs = []
    for o, window in ((out, 0), (out2, 40)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q8.kv8_write(c.cache, batch, k, v)
            q8.kv8_attention(c.cache, batch, q, out=o, window=window, workspace=ws)
        graphs.append(g)
    from tests import kv8_ref as ref
    for step in range(6):
        c.lens += 1
        lens += 1
        (nq, q64), (nk, k64), (nv, v64) = c.rows(8, torch.bfloat16), c.rows(2, torch.bfloat16), c.rows(2, torch.bfloat16)
        q.copy_(nq), k.copy_(nk), v.copy_(nv)
        for codes, scales, x in ((c.k, c.ks, k64), (c.v, c.vs, v64)):
            ref.write(codes, scales, c.table, c.lens, c.starts, x)
        for g in graphs:
            g.replay()
        eager = q8.kv8_attention(c.cache, batch, q)
        torch.cuda.synchronize()
        c.check_attention(q, q64, out)
        c.check_attention(q, q64, out2, window=40)
        assert torch.equal(eager, out)


def test_prompt_then_tokens():
    """A prompt in chunks, then single tokens: each step's outputs against attention over the values that
    the cache then holds."""
    from tests import kv8_ref as ref
    c = Case([(1, 0), (1, 0)], 2, 64, 32, 32, seed=13)
    c.table = np.arange(16, dtype=np.int32).reshape(2, 8)[:, ::-1].copy()
    c.k, c.v = (np.zeros((16, 2, 32, 64), np.int8) for _ in range(2))
    c.ks, c.vs = (np.full((16, 2, 1), np.nan, np.float32) for _ in range(2))
    c.upload()
    for news in ((50, 3), (77, 0), (1, 1), (2, 100), (1, 1)):
        c.lens = c.lens + np.array(news, np.int32)
        c.starts = np.array([0, news[0], sum(news)], np.int32)
        c.n_tok = sum(news)
        c.sizes = list(zip(news, c.lens.tolist()))
        batch = c.make_batch(max_new=max(news))
        (q, q64), (k, k64), (v, v64) = c.rows(4, torch.float16), c.rows(2, torch.float16), c.rows(2, torch.float16)
        for codes, scales, x in ((c.k, c.ks, k64), (c.v, c.vs, v64)):
            ref.write(codes, scales, c.table, c.lens, c.starts, x)
        c.q8.kv8_write(c.cache, batch, k, v)
        out, lse = run(c, q, batch=batch)
        c.check_attention(q, q64, out, lse)


def test_side_stream():
    c = Case([(1, 900), (33, 200)], 2, 128, seed=14).upload()
    q, q64 = c.rows(4, torch.bfloat16)
    want = c.q8.kv8_attention(c.cache, c.batch, q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = c.q8.kv8_attention(c.cache, c.batch, q)
    side.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("splits", [1, 3])
def test_tiled_prompts_in_a_graph(splits):
    """The tiled kernel captured on a side stream and replayed while lengths and starts move, two graphs on
    one workspace, eager work in between; rows behind the last sequence stay."""
    c = Case([(70, 300), (40, 500)], 1, 128, seed=23)
    c.n_tok = 130
    c.upload()
    lens, starts = (torch.from_numpy(a.copy()).cuda() for a in (c.lens, c.starts))
    batch = c.q8.Kv8Batch(c.batch.page_table, lens, starts, n_tok=130, max_new=130)
    q, q64 = c.rows(4, torch.bfloat16)
    ws = torch.empty(splits * 130 * 4 * 129 * 4, dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.empty_like(q) for _ in range(2)], []
    for out, window in zip(outs, (0, 100)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            c.q8.kv8_attention_debug(c.cache, batch, q, 2, splits=splits, window=window, out=out, workspace=ws)
        graphs.append(g)
    for news, lengths in (((70, 40), (300, 500)), ((1, 129), (64, 448)), ((0, 3), (0, 3)), ((128, 1), (290, 1))):
        c.lens, c.starts = np.array(lengths, np.int32), np.array([0, news[0], sum(news)], np.int32)
        lens.copy_(torch.from_numpy(c.lens)), starts.copy_(torch.from_numpy(c.starts))
        n = sum(news)
        for out in outs:
            out.fill_(7)
        for g in graphs:
            g.replay()
        eager = c.q8.kv8_attention_debug(c.cache, batch, q, 2, splits=splits, workspace=ws)
        torch.cuda.synchronize()
        for out, window in zip(outs, (0, 100)):
            assert (out[n:] == 7).all()
            c.check_attention(q[:n], q64[:n], out[:n], window=window)
        assert torch.equal(eager[:n], outs[0][:n])


def test_long_cache_chunk_takes_splits():
    """Few rows over many keys: the tiled kernel with splits, the workspace's size deciding how many."""
    c = Case([(256, 6000)], 4, 64, seed=24).upload()
    q, _ = c.rows(16, torch.bfloat16)
    ws = c.q8.kv8_attention_workspace(c.cache, c.batch, 16)
    one = 256 * 16 * 65 * 4
    assert ws.numel() >= 2 * one and ws.numel() % one == 0
    auto, lse = run(c, q, workspace=ws)
    tiled, lse1 = run(c, q, 2, splits=ws.numel() // one, workspace=ws)
    assert torch.equal(auto, tiled) and torch.equal(lse, lse1)
    vmax = 127 / 60
    for less in (2 * one, 0):
        out, lse1 = run(c, q, workspace=ws[:less])
        assert (out.float() - auto.float()).abs().max() <= 2 * vmax * (2.0 ** -11 + torch.finfo(q.dtype).eps)
        assert (lse1 - lse).abs().max() <= 2.0 ** -12


@both
def test_rows_before_the_first_sequence(kernel):
    """starts[0] above 0 (which the contract excludes): no row outside the sequences is touched, query heads far
    apart, and the sequences' rows come out as ever."""
    c = Case([(40, 200), (9, 90)], 1, 64, seed=25).upload()
    q, q64 = c.rows(3, torch.bfloat16)
    apart = torch.randn(3, 49 + 50, 64, device="cuda").bfloat16()  # [head][token]
    apart[:, 50:] = q.transpose(0, 1)
    qs = apart.transpose(0, 1)
    starts = torch.from_numpy(c.starts + 50).int().cuda()
    b = c.q8.Kv8Batch(c.batch.page_table, c.batch.lens, starts, n_tok=99, max_new=40)
    out, lse = torch.full((99, 3, 64), 7.0, device="cuda", dtype=torch.bfloat16), torch.full((99, 3), 7.0, device="cuda")
    c.q8.kv8_attention_debug(c.cache, b, qs, kernel, out=out, lse=lse)
    torch.cuda.synchronize()
    assert (out[:50] == 7).all() and (lse[:50] == 7).all()
    c.check_attention(q, q64, out[50:], lse[50:])


@both
def test_starts_in_no_order(kernel):
    """Rows of every sequence are read and written within the arrays, whatever starts holds."""
    c = Case([(30, 100), (30, 100), (30, 100)], 1, 64, seed=26).upload()
    q, _ = c.rows(3, torch.bfloat16)
    for starts in ((0, 80, 20, 90), (70, 3, 90, 1), (-5, 500, 60, 30)):
        b = c.q8.Kv8Batch(c.batch.page_table, c.batch.lens, torch.tensor(starts, dtype=torch.int32, device="cuda"), n_tok=90)
        out = torch.empty(92, 3, 64, device="cuda", dtype=torch.bfloat16).fill_(7)
        c.q8.kv8_attention_debug(c.cache, b, q, kernel, out=out[1:91])
        torch.cuda.synchronize()
        assert (out[0] == 7).all() and (out[91] == 7).all()


def test_lse_joins_two_caches():
    """What lse is for: attention over two halves of the keys joined by their sums."""
    c = Case([(1, 256)], 1, 64, 64, seed=15).upload()
    q, q64 = c.rows(4, torch.float32)
    whole, _ = run(c, q)
    parts = []
    for lo in (0, 2):
        b = c.q8.Kv8Batch(c.batch.page_table[:, lo:lo + 2].contiguous(), torch.tensor([128], dtype=torch.int32, device="cuda"))
        parts.append(run(c, q, batch=b))
    w = torch.softmax(torch.stack([l for _, l in parts]), 0)[..., None]
    joined = (w * torch.stack([o for o, _ in parts])).sum(0)
    assert (joined - whole).abs().max() <= 2.0 ** -16 * 2


def test_argument_checks():
    c = Case([(1, 10), (1, 20)], 2, 64).upload()
    q8, q = c.q8, torch.zeros(2, 4, 64, device="cuda")
    k = torch.zeros(2, 2, 64, device="cuda")
    for bad in (q[:1], q[..., :32], q[:, :3], q.transpose(1, 2).contiguous().transpose(1, 2), q.double(), q.cpu(), q[0]):
        with pytest.raises((ValueError, q8.Q8Error)):
            q8.kv8_attention(c.cache, c.batch, bad)
    for kw in (dict(window=-1), dict(scale=float("nan")), dict(sinks=torch.zeros(3, device="cuda")), dict(out=q[:1]),
               dict(sinks=torch.zeros(4, device="cuda").half()), dict(lse=torch.zeros(2, 4)), dict(out_dtype=torch.int8),
               dict(workspace=torch.zeros(8, device="cuda"))):
        with pytest.raises((ValueError, q8.Q8Error)):
            q8.kv8_attention(c.cache, c.batch, q, **kw)
    for bad in (dict(k=k[:, :1], v=k), dict(k=k, v=k.half()), dict(k=k, v=k[:1]), dict(k=k.int(), v=k.int())):
        with pytest.raises((ValueError, q8.Q8Error)):
            q8.kv8_write(c.cache, c.batch, **bad)
    with pytest.raises(ValueError):
        q8.kv8_read(c.cache, c.batch, k=k[:1])
    with pytest.raises(ValueError):
        q8.kv8_read(c.cache, c.batch, torch.int32)
    with pytest.raises(ValueError):
        q8.Kv8Batch(c.batch.page_table, c.batch.lens[:1])
    with pytest.raises(ValueError):
        q8.Kv8Batch(c.batch.page_table, c.batch.lens, c.batch.starts)
    with pytest.raises(ValueError):
        q8.Kv8Batch(c.batch.page_table.long(), c.batch.lens)
    for bad in (dict(d=96), dict(p=48), dict(b=8)):
        s = {**dict(p=64, d=64, b=16), **bad}
        cache = q8.kv8_cache(3, 1, s["d"], s["p"], s["b"])
        with pytest.raises(q8.Q8Error):
            q8.kv8_attention(cache, c.batch, torch.zeros(2, 1, s["d"], device="cuda"))
