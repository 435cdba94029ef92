"""kv8_write, kv8_read and kv8_attention at the edges of what their header allows, and on lengths,
starts and scales that a batch should not have."""
import numpy as np
import pytest
import torch

from tests import kv8_ref as ref
from tests.helpers import say
from tests.kv8_helpers import DTYPES, Case

pytestmark = pytest.mark.gpu


def cache_bytes(c):
    return [t.clone() for t in (c.cache.k, c.cache.v, c.cache.k_scales, c.cache.v_scales)]


@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_write_rows_before_the_first_sequence(block):
    """starts[0] above 0 (which the contract excludes) and sequences with fewer tokens than rows: no page but the
    sequences' own is written, though the words before the table name pages; the sequences' rows come out as ever."""
    say("write, rows before the first sequence", block)
    c = Case([(40, 25), (9, 3), (block + 3, 2)], 2, 64, 128, block, seed=block, spare=5).upload()
    used = set(c.table[c.table >= 0].tolist())
    others = [p for p in range(c.k.shape[0]) if p not in used]
    width = c.table.shape[1]
    table = np.full((4, width), others[0], np.int32)  # the words before the table
    table[1:] = np.where(c.table < 0, others[1], c.table)
    on_device = torch.from_numpy(table).cuda()
    for before in (1, block, 3 * block + 5, 400):
        starts = torch.from_numpy(c.starts + before).int().cuda()
        n_tok = c.n_tok + before
        b = c.q8.Kv8Batch(on_device[1:], c.batch.lens, starts, n_tok=n_tok)
        x = torch.from_numpy(c.rng.standard_normal((n_tok, 2, 64))).float().cuda()
        for codes, scales, sign in ((c.k, c.ks, 1), (c.v, c.vs, -1)):
            ref.write(codes, scales, c.table, c.lens, c.starts, sign * x[before:].double().cpu().numpy())
        c.q8.kv8_write(c.cache, b, x, -x)
        torch.cuda.synchronize()
        for name, got, want in zip(("k", "v", "k scales", "v scales"), c.downloaded(), (c.k, c.v, c.ks, c.vs)):
            assert np.array_equal(got, want), (name, before)


def test_write_starts_in_no_order():
    """Whatever starts and lens hold, pages that no sequence has keep their bytes."""
    c = Case([(30, 20), (30, 100), (30, 7)], 1, 64, 16, seed=31, spare=4).upload()
    used = set(c.table[c.table >= 0].tolist())
    others = [p for p in range(c.k.shape[0]) if p not in used]
    table = np.full((4, c.table.shape[1]), others[0], np.int32)
    table[1:] = np.where(c.table < 0, others[1], c.table)
    on_device = torch.from_numpy(table).cuda()
    was = cache_bytes(c)
    x = torch.randn(90, 1, 64, device="cuda")
    free = torch.tensor(others, device="cuda")
    for starts in ((0, 80, 20, 90), (70, 3, 90, 1), (-5, 500, 60, 30), (90, 60, 30, 0), (33, 90, 90, 90)):
        say("write, starts", starts)
        b = c.q8.Kv8Batch(on_device[1:], c.batch.lens, torch.tensor(starts, dtype=torch.int32, device="cuda"), n_tok=90)
        c.q8.kv8_write(c.cache, b, x, x)
        k, v = c.q8.kv8_read(c.cache, b)
        torch.cuda.synchronize()
        for a, now in zip(was, cache_bytes(c)):
            assert torch.equal(a[free], now[free]), starts


both = pytest.mark.parametrize("kernel", [1, 2])


def largest_seen(c, n_q, window):
    """The largest value that the finite scales of V which a row sees can stand for, [n_tok][n_q][1]."""
    most = np.zeros((c.n_tok, n_q, 1))
    for s, m in enumerate(c.lens):
        scales = np.stack([np.repeat(c.vs[page], c.block, 1) for page in c.table[s, :-(-m // c.page)]], 1)
        scales = np.where(np.isfinite(scales), scales, 0).reshape(c.hkv, -1)
        for i in range(c.starts[s], c.starts[s + 1]):
            pos = m - c.starts[s + 1] + i
            seen = scales[:, max(0, pos - window + 1) if window else 0:pos + 1].max(1)
            most[i, :, 0] = 127 * np.repeat(seen, n_q // c.hkv)
    return most


def check_by_row(c, q, q64, out, window, rows=None):
    """As Case.check_attention, with the absolute part of each row's tolerance from the scales that the row sees: a
    weight is rounded to fp16 in units in which the row's largest one is 2^7 at least and V's scale 2 at most, and
    fp16 is off by 2^-25 at most below its normal numbers, so a key adds 2^-25 * 2 * vmax / 2^7 (also where
    weights are in two halves, the second of which has the same least step)."""
    scale = float(np.float32(1.0 / np.sqrt(c.d)))
    want, _, mag, smag, keys = ref.attention(c.k, c.ks, c.v, c.vs, c.table, c.lens, c.starts, q64, scale, window)
    halves = torch.float32 in (q.dtype, out.dtype)
    vmax = largest_seen(c, q.shape[1], window)
    tol = ref.attention_tolerance(want, mag, smag, keys, c.d, vmax, out.dtype, halves) + vmax * keys[..., None] * 2.0 ** -31
    got = out.double().cpu().numpy()
    if rows is not None:
        got, want, tol = got[rows], want[rows], tol[rows]
    assert np.array_equal(np.isnan(got), np.isnan(want)), "NaN at other places"
    ok = ~np.isnan(want)
    err = np.abs(got - want)[ok] / tol[ok]
    say("worst", err.max())
    assert err.max() <= 1, f"{(err > 1).sum()} of {err.size} outside, worst {err.max():.3g} times the tolerance"


# a scale that a row does not see over those that it sees
UNSEEN = [2.0 ** 12, 2.0 ** 25, 2.0 ** 60, 2.0 ** 125, np.nan, np.inf]


@both
@pytest.mark.parametrize("unseen", UNSEEN)
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (64, "fp32"), (128, "bf16"), (128, "fp32"), (192, "bf16"), (256, "fp32"),
                                     (512, "bf16")])
@pytest.mark.parametrize("where", ["later", "before"])
def test_scales_of_unseen_keys(where, d, dtype, unseen, kernel):
    """Blocks that only later rows of the same tile see, or that lie before a row's window, have scales of V far
    above those that the row sees, or none that is a number."""
    say("unseen scales", where, d, dtype, unseen, kernel)
    window = 20 if where == "before" else 0
    c = Case([(40, 100), (9, 300), (33, 33), (5, 18)], 1, d, 64, 16, seed=d)
    finite = np.isfinite(unseen)
    c.ks[:], c.vs[:] = c.ks / 4, c.vs * np.float32(1.0 if finite else 2.0 ** -40)
    sees = np.zeros(c.n_tok, bool)  # rows that have such a block among their keys
    for s, (n, m) in enumerate(c.sizes):
        blk = (m - 16) // 16 if where == "later" else max(m - n // 2 - window, 0) // 16
        c.vs[c.table[s, blk // 4], 0, blk % 4] *= np.float32(unseen)
        for i in range(n):
            pos = m - n + i
            lo = max(0, pos - window + 1) if window else 0
            sees[c.starts[s] + i] = lo <= 16 * blk + 15 and pos >= 16 * blk
    assert sees.any() and not sees.all()
    c.upload()
    q, q64 = c.rows(3, DTYPES[dtype])
    lse = torch.empty(c.n_tok, 3, device="cuda")
    out = c.q8.kv8_attention_debug(c.cache, c.batch, q, kernel, window=window, lse=lse)
    torch.cuda.synchronize()
    check_by_row(c, q, q64, out, window, None if not np.isinf(unseen) else ~sees)


@both
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("step", [2.0 ** 9, 2.0 ** 25, 2.0 ** -9, 2.0 ** -25])
@pytest.mark.parametrize("window", [0, 20])
def test_scales_that_grow_or_fall_by_block(window, step, dtype, kernel):
    """Each block's scale of V is far from the last one's: every row has an exponent of its own."""
    c = Case([(70, 90), (1, 90), (33, 60)], 1, 64, 16, 16, seed=41)
    c.ks[:] /= 4
    for s, (n, m) in enumerate(c.sizes):
        for blk in range(-(-m // 16)):
            c.vs[c.table[s, blk]] *= np.float32(step ** (blk - 2.5))
    c.upload()
    q, q64 = c.rows(3, DTYPES[dtype])
    out = c.q8.kv8_attention_debug(c.cache, c.batch, q, kernel, window=window)
    torch.cuda.synchronize()
    check_by_row(c, q, q64, out, window)


@both
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 30, 2 ** 30 - 1])
def test_windows_beyond_every_length(window, kernel):
    """A window that no length reaches is none, also in tiles that begin at positions below 0."""
    c = Case([(20, 7), (1, 40), (300, 290), (5, 0)], 1, 64, seed=43).upload()
    q, q64 = c.rows(1, torch.bfloat16)
    lse, lse0 = (torch.empty(c.n_tok, 1, device="cuda") for _ in range(2))
    out = c.q8.kv8_attention_debug(c.cache, c.batch, q, kernel, window=window, lse=lse)
    assert torch.equal(out, c.q8.kv8_attention_debug(c.cache, c.batch, q, kernel, lse=lse0)) and torch.equal(lse, lse0)
    c.check_attention(q, q64, out, lse)
    auto = c.q8.kv8_attention(c.cache, c.batch, q, window=window)
    assert torch.equal(auto, c.q8.kv8_attention(c.cache, c.batch, q))


@both
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_lse_does_not_depend_on_values(d, dtype, splits, kernel):
    """A row that sees a NaN scale of V is NaN, and its log sum is that of its scores; a NaN scale of K makes both NaN."""
    c = Case([(1, 100), (90, 100), (3, 50), (1, 700), (40, 40)], 1, d, 16, 16, seed=44)
    c.vs[c.table[1, 3]] = np.nan   # tokens 48 .. 63
    c.vs[c.table[2, 2]] = np.nan   # tokens 32 .. 47
    c.vs[c.table[3, 20]] = 0.0
    c.vs[c.table[4, 0]] = np.nan
    c.ks[c.table[4, 1]] = np.nan
    c.upload()
    q, q64 = c.rows(3, DTYPES[dtype])
    lse = torch.empty(c.n_tok, 3, device="cuda")
    out = c.q8.kv8_attention_debug(c.cache, c.batch, q, kernel, splits=splits, lse=lse)
    torch.cuda.synchronize()
    c.check_attention(q, q64, out, lse)
    whole, sums = out.isnan().all(-1).all(-1).cpu(), lse.isnan().all(-1).cpu()
    assert whole[39:94].all() and not sums[39:94].any() and not whole[:39].any() and not whole[94]
    assert whole[95:].all() and not sums[95:111].any() and sums[111:].all()


@both
@pytest.mark.parametrize("splits", [1, 2, 5, 8, 9, 40])
@pytest.mark.parametrize("far", [10.0, 3000.0])
def test_nan_values_of_vanishing_weight(far, splits, kernel):
    """A NaN scale of V under keys whose weights vanish in fp32: the rows that see it are NaN, whichever split it falls
    in; zero weights of other blocks add nothing."""
    c = Case([(1, 1300), (3, 1300), (2, 1300)], 1, 64, 16, 16, seed=45)
    c.k[..., 0] = 100
    for s in range(3):
        c.ks[c.table[s, 70:82]] *= np.float32(far)  # tokens from 1120 on: scores far above the others
    c.vs[c.table[0, 3]] = np.nan
    c.vs[c.table[2, 60]] = np.nan
    c.upload()
    q, _ = c.rows(2, torch.float32)
    q = q.abs()
    lse = torch.empty(c.n_tok, 2, device="cuda")
    out = c.q8.kv8_attention_debug(c.cache, c.batch, q, kernel, splits=splits, lse=lse, scale=1.0)
    torch.cuda.synchronize()
    rows = out.isnan().all(-1).all(-1).tolist()
    assert rows == [True, False, False, False, True, True] and out.isnan().any(-1).any(-1).tolist() == rows
    assert lse.isfinite().all()
    if far < 100:
        c.check_attention(q, q.double().cpu().numpy(), out, lse, scale=1.0)


@both
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (64, "fp32"), (128, "bf16"), (128, "fp32"), (192, "bf16"), (256, "bf16"), (512, "bf16")])
def test_unseen_keys_change_no_bit(d, dtype, splits, kernel):
    """Other tokens behind a row, or before its window, whatever they hold, leave its output's and log sum's bits:
    rows of one tile have bounds and exponents of their own."""
    c = Case([(40, 100), (70, 300), (33, 33), (3, 290), (40, 340)], 1, d, 64, 16, seed=46)
    c.ks[:] /= 4
    q = None
    border = [80, 256, 16, 288, 304]  # tokens from here on change
    kept = [(k.copy(), v.copy()) for k, v in ((c.k, c.ks), (c.v, c.vs))]
    for window in (0, 20):
        before = window > 0  # those before the border change
        want = None
        for what in range(7):
            for (codes, scales), (k0, s0), which in (((c.k, c.ks), kept[0], "k"), ((c.v, c.vs), kept[1], "v")):
                codes[:], scales[:] = k0, s0
                for s, (n, m) in enumerate(c.sizes):
                    for blk in (range(border[s] // 16) if before else range(border[s] // 16, -(-m // 16))):
                        at = (c.table[s, blk // 4], 0, blk % 4)
                        if what == 1:
                            scales[at] *= np.float32(60.0) if which == "k" else np.float32(1.0)  # scores far above
                        elif what == 2:
                            scales[at] *= np.float32(2.0 ** 100) if which == "v" else np.float32(1.0)
                        elif what == 3:
                            scales[at] = 0
                        elif what == 4:
                            scales[at] = np.nan
                        elif what == 5:
                            scales[at] *= np.float32(2.0 ** -30)
                        elif what == 6:
                            page = codes[at[0], 0, 16 * at[2]:16 * at[2] + 16]
                            page[:] = c.rng.integers(-127, 128, page.shape)
            c.upload()
            if q is None:
                q, _ = c.rows(3, DTYPES[dtype], spread=2.0)
            lse = torch.empty(c.n_tok, 3, device="cuda")
            out = c.q8.kv8_attention_debug(c.cache, c.batch, q, kernel, splits=splits, window=window, lse=lse)
            torch.cuda.synchronize()
            rows = []
            for s, (n, m) in enumerate(c.sizes):
                pos = np.arange(m - n, m)
                rows.append(pos - window + 1 >= border[s] if before else pos < border[s])
            rows = torch.from_numpy(np.concatenate(rows)).cuda()
            assert rows.any() and not rows.all()
            got = out[rows], lse[rows]
            assert got[0].isfinite().all() and got[1].isfinite().all()
            if want is None:
                want = got
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (window, what)
