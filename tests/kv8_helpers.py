"""Caches and ragged batches of the 8-bit key/value cache for the GPU tests: the same
contents as numpy arrays (row-major) and on the device."""
from __future__ import annotations

import numpy as np
import torch

from tests import kv8_ref as ref

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


class Case:
    """sizes: (new rows, length) of each sequence.  Pages in random order; entries behind a sequence's
    length are no pages at all.  The pool is full of codes, unused pages included."""

    def __init__(self, sizes, hkv, d, page=64, block=16, seed=0, one_row=False, spare=2, stale=None):
        import q8_quantized_matmul_amd as q8
        rng = np.random.default_rng(seed)
        self.rng, self.q8 = rng, q8
        self.sizes, self.hkv, self.d, self.page, self.block = sizes, hkv, d, page, block
        self.lens = np.array([m for _, m in sizes], np.int32)
        self.starts = np.concatenate([[0], np.cumsum([n for n, _ in sizes])]).astype(np.int32)
        self.n_tok = int(self.starts[-1])
        used = [-(-max(m, 0) // page) for _, m in sizes]
        n_pages = sum(used) + spare
        order = rng.permutation(n_pages).astype(np.int32)
        self.table = np.full((len(sizes), max(used) + 1), -77, np.int32)
        at = 0
        for s, u in enumerate(used):
            self.table[s, :u] = order[at:at + u]
            at += u
        shape = (n_pages, hkv, page, d)
        self.k, self.v = (rng.integers(-127, 128, shape).astype(np.int8) for _ in range(2))
        self.ks, self.vs = ((rng.uniform(0.3, 1.0, shape[:2] + (page // block,)) / 60).astype(np.float32)
                            for _ in range(2))
        if stale is not None:  # scales of tokens that no sequence holds
            for s in [self.ks, self.vs]:
                live = np.zeros(s.shape, bool)
                for i, m in enumerate(self.lens):
                    for blk in range(-(-max(m, 0) // block)):
                        live[self.table[i, blk * block // page], :, blk * block % page // block] = True
                s[~live] = stale
        self.one_row = one_row

    def upload(self):
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.cache = self.q8.Kv8Cache(dev(ref.k_tiles(self.k)), dev(ref.v_tiles(self.v)), dev(self.ks), dev(self.vs))
        self.batch = self.make_batch()
        return self

    def make_batch(self, **more):
        table, lens, starts = (torch.from_numpy(a.copy()).cuda() for a in (self.table, self.lens, self.starts))
        if self.one_row:
            return self.q8.Kv8Batch(table, lens, **more)
        return self.q8.Kv8Batch(table, lens, starts, n_tok=self.n_tok, **more)

    def downloaded(self):
        """(k codes, v codes, k scales, v scales) of the device, row-major."""
        c = self.cache
        return (ref.k_rows(c.k.cpu().numpy()), ref.v_rows(c.v.cpu().numpy()), c.k_scales.cpu().numpy(), c.v_scales.cpu().numpy())

    def rows(self, heads, dtype, spread=1.0):
        """(device tensor [n_tok][heads][d], its values in float64)."""
        x = torch.from_numpy(self.rng.standard_normal((self.n_tok, heads, self.d)) * spread).to(dtype)
        return x.cuda(), x.double().numpy()

    def check_attention(self, q, q64, out, lse=None, scale=None, window=0, sinks=None, rows=None):
        """Compares with the 64-bit form; rows: of the batch, those looked at (all)."""
        scale = float(np.float32(1.0 / np.sqrt(self.d) if scale is None else scale))
        want, want_lse, mag, smag, keys = ref.attention(
            self.k, self.ks, self.v, self.vs, self.table, self.lens, self.starts, q64, scale, window,
            None if sinks is None else sinks.double().cpu().numpy())
        halves = q.dtype == torch.float32 or out.dtype == torch.float32
        vmax = 127 * float(np.nanmax(np.where(np.isfinite(self.vs), self.vs, 0)))
        tol = ref.attention_tolerance(want, mag, smag, keys, self.d, vmax, out.dtype, halves)
        got = out.double().cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(want)), "NaN at other places"
        ok = ~np.isnan(want)
        err = np.abs(got - want)[ok] / tol[ok]
        assert err.size == 0 or err.max() <= 1, f"{(err > 1).sum()} of {err.size} outside, worst {err.max():.3g} times the tolerance"
        if lse is not None:
            g = lse.double().cpu().numpy()
            tl = ref.lse_tolerance(want_lse, smag, keys, self.d)
            assert np.array_equal(np.isnan(g), np.isnan(want_lse))
            fin = np.isfinite(want_lse)
            assert np.array_equal(g[~fin & ~np.isnan(g)], want_lse[~fin & ~np.isnan(g)])
            assert (np.abs(g - want_lse)[fin] <= tl[fin]).all()
        return float(err.max()) if err.size else 0.0
