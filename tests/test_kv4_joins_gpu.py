"""Attention over the paged 4-bit cache, items that many CTAs share: the join of up to 16 partials, and of more, in
every form (channels, rows of a chunk)."""
import pytest

from gpu_util import need_gpu
from test_kv4_gpu import FMTS, Batch

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from block_quantized_gemv_nt_gb300 import nt  # noqa: E402


@pytest.fixture(scope="module")
def ctx():
    need_gpu()
    c = nt.Context(0)
    yield c
    c.close()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("n,H,G,rows", [(70000, 1, 4, 1), (40000, 2, 8, 3), (40000, 1, 3, 2), (30000, 3, 1, 1), (20000, 2, 16, 5)])
def test_many_partials(ctx, fmt, hd, n, H, G, rows):
    b = Batch(ctx, fmt, hd, H, G, [n], [rows], seed=hd + G)
    b.check(b.run())
    ctx.sync()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("G", [4, 8])                   # chunks of 4 and of 8 rows
@pytest.mark.parametrize("pages", [120, 127, 128, 129, 136, 137])
def test_sixteen_and_seventeen_partials(ctx, fmt, hd, G, pages):
    """A page a warp, 8 warps a CTA: an item of 128 pages is 16 CTAs', of 129 it is 17's, the second head's begun in the
    middle of one.  (The table is too wide for a cluster of their own.)"""
    b = Batch(ctx, fmt, hd, 2, G, [64 * pages - 5], [1], seed=pages, width=200)
    b.check(b.run())
    ctx.sync()


def test_items_of_few_and_many_partials_in_one_call(ctx):
    b = Batch(ctx, nt.KV4_E2M1, 64, 2, 8, [40000, 70, 9000, 0, 64, 20001], [3, 1, 2, 1, 8, 1], seed=21)
    first = b.run()
    b.check(first)
    for _ in range(3):
        assert torch.equal(b.run(), first)
    ctx.sync()
