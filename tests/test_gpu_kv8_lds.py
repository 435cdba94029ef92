"""The 8-bit cache's calls after the LDS of every compute unit was filled with a pattern (as
the Q8_0 and MXFP4 calls' tests do): every run equals the first bit for bit, so no kernel reads LDS
before it is written, or before the barrier that publishes another wave's writes."""
import pytest
import torch

from tests.helpers import say
from tests.kv8_helpers import DTYPES, Case

pytestmark = pytest.mark.gpu

PATTERNS = [0x00000000, 0xFFFFFFFF, 0x7F7F7F7F, 0x80000001, 0x3C00BC00]


def same_after_every_pattern(q8, call):
    first = [o.clone() for o in call()]
    for o in first:
        assert not torch.isnan(o.float()).any()
    for pattern in PATTERNS:
        q8.q8_0_debug_poison_lds(pattern)
        for a, b in zip(first, call()):
            assert torch.equal(a, b), hex(pattern)


@pytest.mark.parametrize("kernel,splits", [(1, 1), (1, 5), (1, 20), (2, 1), (2, 3)])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (64, "fp32"), (128, "fp16"), (128, "fp32"), (192, "bf16"), (192, "fp32"),
                                     (256, "bf16"), (256, "fp32"), (512, "bf16"), (512, "fp32")])
def test_attention(d, dtype, kernel, splits):
    """Tiles of rows that a sequence fills and does not, keys behind the last row, a window, sinks."""
    say("lds, attention", d, dtype, kernel, splits)
    if kernel == 2 and d == 512 and dtype == "fp32":
        pytest.skip("the tiled kernel has no such variant")
    c = Case([(300, 300), (1, 333), (77, 500), (3, 2)], 2, d, seed=d + splits).upload()
    q, _ = c.rows(6, DTYPES[dtype])
    sinks = torch.randn(6, device="cuda")
    for window in (0, 70):
        def call():
            lse = torch.zeros(c.n_tok, 6, device="cuda")
            out = c.q8.kv8_attention_debug(c.cache, c.batch, q, kernel, splits=splits, window=window, sinks=sinks, lse=lse)
            return out, lse.clamp(min=-1e30)
        same_after_every_pattern(c.q8, call)


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "fp32"), (512, "fp16")])
def test_write_and_read(d, dtype, block):
    c = Case([(1, 77), (200, 300), (33, 33)], 3, d, 128, block, seed=block).upload()
    k, _ = c.rows(3, DTYPES[dtype], spread=4.0)
    v, _ = c.rows(3, DTYPES[dtype])
    arrays = c.cache.k, c.cache.v, c.cache.k_scales, c.cache.v_scales
    was = [a.clone() for a in arrays]

    def call():
        for a, b in zip(arrays, was):
            a.copy_(b)
        c.q8.kv8_write(c.cache, c.batch, k, v)
        return *(a.clone() for a in arrays), *c.q8.kv8_read(c.cache, c.batch, DTYPES[dtype])
    same_after_every_pattern(c.q8, call)
