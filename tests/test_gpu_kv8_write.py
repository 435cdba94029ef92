"""kv8_write and kv8_read against their plain 64-bit forms: codes, scales and untouched
bytes bit for bit."""
import numpy as np
import pytest
import torch

from tests import kv8_ref as ref
from tests.helpers import say
from tests.kv8_helpers import DTYPES, Case

pytestmark = pytest.mark.gpu


def check_write(c, k, k64, v, v64, batch=None):
    for codes, scales, x in ((c.k, c.ks, k64), (c.v, c.vs, v64)):
        ref.write(codes, scales, c.table, c.lens, c.starts, x)
    c.q8.kv8_write(c.cache, batch or c.batch, k, v)
    torch.cuda.synchronize()
    for name, got, want in zip(("k", "v", "k scales", "v scales"), c.downloaded(), (c.k, c.v, c.ks, c.vs)):
        same = (got == want) | (np.isnan(got) & np.isnan(want) if got.dtype == np.float32 else False)
        assert same.all(), f"{name}: {(~same).sum()} of {same.size} differ, first at {np.argwhere(~same)[0]}"


SIZES = {
    "one": [(1, 1)],
    "whole": [(64, 64)],
    "ragged": [(5, 5), (1, 40), (0, 9), (33, 100), (130, 131), (16, 32), (1, 17), (64, 129)],
    "decode": [(1, 1), (1, 16), (1, 17), (1, 333), (1, 64), (1, 65)],
    "behind": [(3, 2), (1, 0), (7, 7), (20, -5)],  # rows at negative positions
}


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("d,hkv", [(64, 3), (128, 2), (192, 1), (256, 2), (512, 1)])
@pytest.mark.parametrize("sizes", list(SIZES))
def test_write_read(sizes, d, hkv, dtype):
    say("write", sizes, d, hkv, dtype)
    c = Case(SIZES[sizes], hkv, d, seed=d).upload()
    k, k64 = c.rows(hkv, DTYPES[dtype])
    v, v64 = c.rows(hkv, DTYPES[dtype], spread=1e-3)
    check_write(c, k, k64, v, v64)
    gk, gv = c.q8.kv8_read(c.cache, c.batch, DTYPES[dtype])
    for got, codes, scales in ((gk, c.k, c.ks), (gv, c.v, c.vs)):
        for s, (n, m) in enumerate(c.sizes):
            all_rows = ref.sequence(codes, scales, c.table[s], max(m, 0))
            want = np.zeros((n, hkv, d))
            have = min(n, max(m, 0))
            want[n - have:] = all_rows[max(m, 0) - have:]
            # the product is rounded to fp32 and then to the type
            want = torch.from_numpy(want.astype(np.float32)).to(DTYPES[dtype])
            assert torch.equal(got[c.starts[s]:c.starts[s + 1]].cpu(), want)


@pytest.mark.parametrize("page,block", [(16, 16), (32, 16), (32, 32), (64, 64), (128, 128), (256, 64), (1024, 128)])
def test_pages_and_blocks(page, block):
    c = Case([(70, 300), (1, 150), (257, 257), (1, 129)], 2, 64, page, block, seed=page).upload()
    k, k64 = c.rows(2, torch.bfloat16)
    v, v64 = c.rows(2, torch.bfloat16)
    check_write(c, k, k64, v, v64)


@pytest.mark.parametrize("block", [16, 64, 128])
def test_appends_one_by_one(block):
    """Tokens of growing and shrinking size into a block: its scale only grows, older codes follow."""
    c = Case([(1, 1), (1, 50)], 2, 128, 128, block, one_row=True, seed=3)
    c.lens[:] = (0, 49)
    for step in range(block + 5):
        c.lens += 1
        if step == 0:
            c.upload()
        k, k64 = c.rows(2, torch.float16, spread=2.0 ** c.rng.integers(-3, 4))
        v, v64 = c.rows(2, torch.float16, spread=1.0 + 0.1 * step)
        check_write(c, k, k64, v, v64, c.make_batch())


def test_ties_are_even():
    """Quotients at, and next to, halves: the scale is exactly 2^-3 and 3 * 2^-5."""
    for scale in (2.0 ** -3, 3 * 2.0 ** -5):
        c = Case([(16, 16)], 1, 64, 16).upload()
        x = ((c.rng.integers(-126, 126, (16, 1, 64)) + 0.5) * scale).astype(np.float32)
        x[::3] = np.nextafter(x[::3], np.float32(np.inf))
        x[1::3] = np.nextafter(x[1::3], np.float32(-np.inf))
        x[0, 0, 0] = 127 * scale
        t = torch.from_numpy(x).cuda()
        check_write(c, t, x.astype(np.float64), -t, -x.astype(np.float64))


def test_growth_ties():
    """Older codes at exact halves of the grown scale."""
    c = Case([(1, 9)], 1, 64, 16)
    c.ks[:], c.vs[:] = 2.0 ** -5, 2.0 ** -5
    c.upload()
    x = np.full((1, 1, 64), 127 * 2.0 ** -4)
    t = torch.from_numpy(x).float().cuda()
    check_write(c, t, x, t * 3, x * 3)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_not_finite(value):
    c = Case([(20, 40), (1, 5)], 2, 64).upload()
    k, _ = c.rows(2, torch.float32)
    v, _ = c.rows(2, torch.float32)
    k[13, 1, 5] = value
    v[20, 0, 63] = value
    check_write(c, k, k.double().cpu().numpy(), v, v.double().cpu().numpy())
    # a later token cannot mend the block, its first token written anew does
    k, k64 = c.rows(2, torch.float32)
    v, v64 = c.rows(2, torch.float32)
    check_write(c, k, k64, v, v64)
    c.lens[1] = 1
    check_write(c, k, k64, v, v64, c.make_batch())


def test_zeros_and_small_numbers():
    """All-zero blocks (scale 0), scales below fp32's normal numbers, and ones that vanish."""
    for spread in (0.0, 1e-37, 1e-40, 3e-43, 1e-44, 1e38):
        c = Case([(16, 16), (3, 20)], 1, 64, 16)
        if spread < 1:
            c.ks[:], c.vs[:] = 0.0, 1e-42
        c.upload()
        k, _ = c.rows(1, torch.float32)
        k = (k.clamp(-3, 3) * spread).contiguous()
        k64 = k.cpu().numpy().astype(np.float64)
        check_write(c, k, k64, k, k64)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_strided_rows(dtype, offset):
    """Slices of a fused projection, aligned to 16 bytes and not; heads before tokens."""
    c = Case([(30, 77), (1, 4)], 2, 64).upload()
    x, x64 = c.rows(7, DTYPES[dtype])
    flat = torch.zeros(c.n_tok, 7 * 64 + 24, dtype=DTYPES[dtype], device="cuda")
    flat[:, offset:offset + 7 * 64] = x.view(c.n_tok, -1)
    rows = flat[:, offset:offset + 7 * 64].unflatten(1, (7, 64))
    by_head = x[:, 4:6].transpose(0, 1).contiguous().transpose(0, 1)
    check_write(c, rows[:, 2:4], x64[:, 2:4], by_head, x64[:, 4:6])


def test_bad_pages_are_skipped():
    c = Case([(40, 200), (1, 5), (100, 100)], 2, 64)
    c.table[0, 2] = c.k.shape[0]
    c.table[1, 0] = -1
    c.table[2, 0] = 2 ** 31 - 1
    c.upload()
    k, k64 = c.rows(2, torch.bfloat16)
    v, v64 = c.rows(2, torch.bfloat16)
    check_write(c, k, k64, v, v64)
    gk, gv = c.q8.kv8_read(c.cache, c.batch, torch.bfloat16)
    for got, codes, scales in ((gk, c.k, c.ks), (gv, c.v, c.vs)):
        for s, (n, m) in enumerate(c.sizes):
            want = torch.from_numpy(ref.sequence(codes, scales, c.table[s], m)[m - n:].astype(np.float32)).bfloat16()
            assert torch.equal(torch.nan_to_num(got[c.starts[s]:c.starts[s + 1]].cpu(), nan=99), torch.nan_to_num(want, nan=99))


def test_lengths_beyond_the_table_are_held():
    """lens and starts out of their ranges stay within the buffers."""
    c = Case([(4, 60), (4, 64)], 1, 64, spare=0).upload()
    k, _ = c.rows(1, torch.float32)
    table, starts = torch.from_numpy(c.table[:, :1].copy()).cuda(), torch.from_numpy(c.starts).cuda()
    for lens, st in (([2 ** 31 - 1, 64], starts), ([60, 64], starts * 100), ([60, -2 ** 31], starts - 5)):
        b = c.q8.Kv8Batch(table, torch.tensor(lens, dtype=torch.int32).cuda(), st, n_tok=8)
        c.q8.kv8_write(c.cache, b, k, k)
        c.q8.kv8_read(c.cache, b)
        c.q8.kv8_attention(c.cache, b, k)
    torch.cuda.synchronize()


def test_rows_behind_the_last_sequence():
    c = Case([(3, 30), (2, 2)], 2, 64)
    c.upload()
    table, lens, starts = (torch.from_numpy(a).cuda() for a in (c.table, c.lens, c.starts))
    b = c.q8.Kv8Batch(table, lens, starts, n_tok=9, max_new=3)
    out = torch.full((9, 2, 64), 7.0, device="cuda")
    gk, gv = c.q8.kv8_read(c.cache, b, k=out, v=out.clone())
    assert gk is out and (gk[5:] == 7).all() and (gv[5:] == 7).all() and not (gk[:5] == 7).all()


@pytest.mark.parametrize("which", ["k", "v"])
def test_read_one_of_two(which):
    from q8_quantized_matmul_amd import kv8
    c = Case([(37, 37)], 3, 64).upload()
    both = dict(zip("kv", c.q8.kv8_read(c.cache, c.batch)))
    out = torch.empty_like(both[which])
    ptr = {"k": None, "v": None, which: out.data_ptr()}
    assert c.q8.raw_library().kv8_read(c.cache._ref, c.batch._ref, ptr["k"], ptr["v"], kv8.KV8_F32,
                                       torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(out, both[which])


def test_many_sequences():
    """More sequences than a wave has lanes, and than its square."""
    rng = np.random.default_rng(0)
    for n_seq in (65, 5000):
        sizes = [(int(n), int(n + m)) for n, m in zip(rng.integers(0, 4, n_seq), rng.integers(0, 20, n_seq))]
        c = Case(sizes, 1, 64, 16, spare=1).upload()
        k, k64 = c.rows(1, torch.bfloat16)
        v, v64 = c.rows(1, torch.bfloat16)
        check_write(c, k, k64, v, v64, c.make_batch(max_new=3))
