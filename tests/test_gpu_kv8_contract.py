"""kv8_write, kv8_read and kv8_attention at the edges of what their header allows, and on lengths,
starts and scales that a batch should not have."""
import numpy as np
import pytest
import torch

from tests import kv8_ref as ref
from tests.helpers import say
from tests.kv8_helpers import Case

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
