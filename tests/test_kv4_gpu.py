"""The paged 4-bit KV cache on the GPU against the 64-bit numpy oracle (kv4_ref):
writing and reading rows, the attention over pages, whole steps, refusals."""
import numpy as np
import pytest

import kv4_ref as ref
from gpu_util import dev, host, need_gpu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from block_quantized_gemv_nt_gb300 import engine, nt  # noqa: E402

FMTS = [nt.KV4_I4, nt.KV4_E2M1]


@pytest.fixture(scope="module")
def ctx():
    need_gpu()
    c = nt.Context(0)
    yield c
    c.close()


def _rows(rng, n, H, hd, spread=0.5):
    return (rng.standard_normal((n, H, hd)) * np.exp(spread * rng.standard_normal((H, hd)))).astype(np.float32)


def _slots(rng, n_pages, n, start=0):
    page = rng.permutation(n_pages)
    i = np.arange(start, start + n)
    return page[i // 64] * 64 + i % 64, page.astype(np.int32)


def _written(ctx, fmt, rows_k, rows_v, slots, n_pages, dtype=torch.float32, cache=None):
    H, hd = rows_k.shape[1:]
    cache = cache or engine.KV4Cache(ctx, fmt, H, hd, n_pages)
    cache.append(dev(rows_k, dtype), dev(rows_v, dtype), dev(slots, torch.int64))
    return cache


# ---- writing and reading ---------------------------------------------------------
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("H,n", [(1, 1), (3, 5), (2, 200), (8, 67)])
def test_rows_come_back_as_the_oracle_says(ctx, fmt, hd, dtype, H, n):
    rng = np.random.default_rng(n * 7 + H)
    k, v = (_rows(rng, n, H, hd).astype(np.float16).astype(np.float32) if dtype is torch.float16 else _rows(rng, n, H, hd)
            for _ in range(2))
    slots, _ = _slots(rng, 6, n, 13)
    cache = _written(ctx, fmt, k, v, slots, 6, dtype)
    for out_type in (torch.float32, torch.float16):
        ko, vo = (torch.empty(n, H, hd, dtype=out_type, device="cuda") for _ in range(2))
        cache.read(ko, vo, dev(slots, torch.int64))
        assert np.array_equal(host(ko).astype(np.float64), ref.values(k, fmt))
        assert np.array_equal(host(vo).astype(np.float64), ref.values(v, fmt))
    ctx.sync()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("scale", [1.0, 0.0117, 2.0 ** -19, 2.0 ** -24, 2.0 ** -26, 171.0, 2500.0, 1e5, 1e30])
def test_borders_of_the_codes(ctx, fmt, scale):
    """Values on, and one step to either side of, every border between two codes."""
    top = 8.0 if fmt == nt.KV4_I4 else 6.0
    borders = np.arange(-8, 9) + 0.5 if fmt == nt.KV4_I4 else np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.0])
    rows = []
    for sign in (1.0, -1.0):
        for b in borders:
            for hit in (-1, 0, 1):
                g = np.zeros(32, dtype=np.float32)
                g[0] = np.float32(sign * top * scale)
                d = float(ref.scales(g.astype(np.float64)[None], fmt)[0])
                for j, s in enumerate((1.0, -1.0)):
                    x = np.float32(s * b * d)
                    if hit:
                        x = np.nextafter(x, np.float32(np.inf * hit))
                    if abs(x) <= abs(g[0]):
                        g[1 + j] = x
                rows.append(g)
    rows = np.stack(rows)
    rows = rows[:len(rows) // 4 * 4].reshape(-1, 1, 128)
    n = rows.shape[0]
    cache = _written(ctx, fmt, rows, -rows, np.arange(n), 4)
    ko, vo = (torch.empty(n, 1, 128, device="cuda") for _ in range(2))
    cache.read(ko, vo, dev(np.arange(n), torch.int64))
    assert np.array_equal(host(ko), ref.values(rows, fmt).astype(np.float32))
    assert np.array_equal(host(vo), ref.values(-rows, fmt).astype(np.float32))
    ctx.sync()


@pytest.mark.parametrize("fmt", FMTS)
def test_scales_halfway_between_two(ctx, fmt):
    """The largest values whose quotient lies at, or next to, the middle of two scales."""
    mids = (np.arange(128, 256) + 0.5) / 64
    rows = []
    for m in mids:
        for hit in (-1, 0, 1):
            x = np.float32(m * (8.0 if fmt == nt.KV4_I4 else 6.0))
            x = np.nextafter(x, np.float32(np.inf * hit)) if hit else x
            g = np.linspace(-0.97, 0.97, 32).astype(np.float32) * x
            g[5] = x
            rows.append(g)
    rows = np.stack(rows).reshape(-1, 3, 128)
    n = rows.shape[0]
    cache = _written(ctx, fmt, rows, rows, np.arange(n), 2)
    ko, vo = (torch.empty(n, 3, 128, device="cuda") for _ in range(2))
    cache.read(ko, vo, dev(np.arange(n), torch.int64))
    assert np.array_equal(host(ko), ref.values(rows, fmt).astype(np.float32))
    assert np.array_equal(host(vo), ref.values(rows, fmt).astype(np.float32))


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_that_are_not_finite(ctx, fmt):
    rng = np.random.default_rng(3)
    k = _rows(rng, 6, 2, 64)
    k[0, 0, 3], k[1, 0, 40], k[2, 1, 5], k[3, 1, 6:9] = np.nan, np.inf, -np.inf, [np.inf, np.nan, -np.inf]
    k[4, 0, :32] = np.nan
    k[4, 1, :32] = 0
    k[4, 1, 7] = np.inf
    v = _rows(rng, 6, 2, 64)
    cache = _written(ctx, fmt, k, v, np.arange(6), 1)
    ko, vo = (torch.empty(6, 2, 64, device="cuda") for _ in range(2))
    cache.read(ko, vo, dev(np.arange(6), torch.int64))
    assert np.array_equal(host(ko), ref.values(k, fmt).astype(np.float32))
    assert np.array_equal(host(vo), ref.values(v, fmt).astype(np.float32))
    with pytest.raises(nt.NtError, match="4-bit"):
        ctx.sync()
    ctx.sync()


@pytest.mark.parametrize("fmt", FMTS)
def test_slots_left_out_and_behind_the_cache(ctx, fmt):
    rng = np.random.default_rng(4)
    n, H, hd, n_pages = 9, 2, 128, 3
    k, v = _rows(rng, n, H, hd), _rows(rng, n, H, hd)
    pool = torch.full((n_pages + 2, H, nt.nt_kv4_layout(hd)), 0x5A, dtype=torch.uint8, device="cuda")
    cache = engine.KV4Cache(ctx, fmt, H, hd, n_pages, data=pool[1:-1])
    slots = np.array([5, -1, 64 * 3 - 1, -7, 64 * 3, 70, 1 << 40, -(1 << 40), 0])
    cache.append(dev(k), dev(v), dev(slots, torch.int64))
    with pytest.raises(nt.NtError, match="slot"):
        ctx.sync()
    ko, vo = (torch.full((n, H, hd), 7.5, device="cuda") for _ in range(2))
    cache.read(ko, vo, dev(slots, torch.int64))
    with pytest.raises(nt.NtError, match="slot"):
        ctx.sync()
    there = (slots >= 0) & (slots < 64 * n_pages)
    assert np.array_equal(host(ko)[there], ref.values(k, fmt)[there].astype(np.float32))
    assert np.array_equal(host(vo)[there], ref.values(v, fmt)[there].astype(np.float32))
    assert (host(ko)[~there] == 7.5).all() and (host(vo)[~there] == 7.5).all()
    assert (host(pool[0]) == 0x5A).all() and (host(pool[-1]) == 0x5A).all()
    # nothing else of the pages changed: as many bytes as the four rows and their scales have
    assert (host(pool[1:-1]) != 0x5A).sum() <= 4 * H * 2 * (hd // 2 + hd // 16)


def test_a_row_written_again_and_its_neighbours(ctx):
    rng = np.random.default_rng(5)
    k, v = _rows(rng, 64, 2, 64), _rows(rng, 64, 2, 64)
    cache = _written(ctx, nt.KV4_I4, k, v, np.arange(64), 1)
    k[17], v[17] = 100 * _rows(rng, 1, 2, 64)[0], 0
    cache.append(dev(k[17:18]), dev(v[17:18]), torch.tensor([17], device="cuda"))
    ko, vo = (torch.empty(64, 2, 64, device="cuda") for _ in range(2))
    cache.read(ko, vo, torch.arange(64, device="cuda"))
    assert np.array_equal(host(ko), ref.values(k, 0).astype(np.float32))
    assert np.array_equal(host(vo), ref.values(v, 0).astype(np.float32))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_strides(ctx, dtype):
    """Rows of a fused QKV buffer, and rows laid out by heads."""
    rng = np.random.default_rng(6)
    n, H, hd = 70, 3, 64
    qkv = torch.from_numpy(_rows(rng, n, 5 * H, hd)).to(dtype).cuda()
    k, v = qkv[:, 3 * H:4 * H], qkv[:, 4 * H:]
    slots = torch.arange(3, 3 + n, device="cuda")
    cache = engine.KV4Cache(ctx, nt.KV4_E2M1, H, hd, 2)
    cache.append(k, v, slots)
    by_head = torch.zeros(2, H, n + 2, hd, dtype=dtype, device="cuda")
    ko, vo = (by_head[i, :, 1:1 + n].transpose(0, 1) for i in range(2))
    cache.read(ko, vo, slots)
    assert np.array_equal(host(ko).astype(np.float64), ref.values(host(k), 1))
    assert np.array_equal(host(vo).astype(np.float64), ref.values(host(v), 1))
    assert (host(by_head[:, :, 0]) == 0).all() and (host(by_head[:, :, -1]) == 0).all()
    again = engine.KV4Cache(ctx, nt.KV4_E2M1, H, hd, 2)
    again.append(ko, vo, slots)                  # values of the cache quantise to themselves where the scale is kept
    k2, v2 = torch.empty(n, H, hd, device="cuda"), torch.empty(n, H, hd, device="cuda")
    again.read(k2, v2, slots)
    assert np.array_equal(host(k2), ref.values(host(ko), 1).astype(np.float32))


def test_one_of_k_and_v_read(ctx):
    rng = np.random.default_rng(7)
    k, v = _rows(rng, 5, 1, 64), _rows(rng, 5, 1, 64)
    cache = _written(ctx, nt.KV4_I4, k, v, np.arange(5), 1)
    out, s = torch.empty(5, 1, 64, device="cuda"), torch.arange(5, device="cuda")
    nt.nt_kv4_read(ctx, cache.desc, nt.F32, None, out, 5, 64, 64, s)
    assert np.array_equal(host(out), ref.values(v, 0).astype(np.float32))
    nt.nt_kv4_read(ctx, cache.desc, nt.F32, out, None, 5, 64, 64, s)
    assert np.array_equal(host(out), ref.values(k, 0).astype(np.float32))


# ---- attention -------------------------------------------------------------------
class Batch:
    """Requests of the given lengths and row counts over one cache with pages in random order."""

    def __init__(self, ctx, fmt, hd, H, G, held, rows, seed=0, garbage=0xFF, spread=0.5, q_size=1.5, width=0):
        rng = np.random.default_rng(seed)
        self.held, self.rows, self.fmt = held, rows, fmt
        used = [-(-n // 64) for n in held]
        n_pages = sum(used) + 2
        order = rng.permutation(n_pages).astype(np.int32)
        W = max(1, width, *used)
        table = np.full((len(held), W), -5, dtype=np.int32)     # entries behind a request's pages are never read
        self.k, self.v, slots, at = [], [], [], 0
        for r, n in enumerate(held):
            table[r, :used[r]] = order[at:at + used[r]]
            at += used[r]
            p = np.arange(n)
            slots.append(table[r, p // 64].astype(np.int64) * 64 + p % 64)
            self.k.append(_rows(rng, n, H, hd, spread))
            self.v.append(_rows(rng, n, H, hd, spread))
        # what was never written is whatever the memory holds: NaN scales among it
        data = torch.full((n_pages, H, nt.nt_kv4_layout(hd)), garbage, dtype=torch.uint8, device="cuda")
        self.cache = engine.KV4Cache(ctx, fmt, H, hd, n_pages, data=data)
        if sum(held):
            self.cache.append(dev(np.concatenate(self.k)), dev(np.concatenate(self.v)), dev(np.concatenate(slots)))
        self.table, self.held_dev = dev(table), dev(np.array(held, dtype=np.int32))
        self.q_start = dev(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32))
        self.q = (q_size * rng.standard_normal((sum(rows), H * G, hd))).astype(np.float32)

    def run(self, pad=0):
        q = np.concatenate([self.q, np.zeros((pad,) + self.q.shape[1:], dtype=np.float32)])
        out = torch.full(q.shape, 123.0, device="cuda")
        self.cache.attend(dev(q), out, self.q_start, self.held_dev, self.table)
        return out

    def expect(self):
        outs, bounds, at = [], [], 0
        for k, v, n in zip(self.k, self.v, self.rows):
            o, b = ref.attend(self.q[at:at + n], ref.values(k, self.fmt), ref.values(v, self.fmt), n)
            outs.append(o), bounds.append(b)
            at += n
        return np.concatenate(outs), np.concatenate(bounds)

    def check(self, got):
        want, bound = self.expect()
        off = np.abs(host(got)[:len(want)].astype(np.float64) - want)
        assert (off <= bound).all(), (float((off / bound).max()), np.argwhere(off > bound)[:3])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("G", [1, 3, 4, 8, 16])
@pytest.mark.parametrize("n", [1, 63, 64, 65, 130, 1088])
def test_one_request(ctx, fmt, hd, G, n):
    b = Batch(ctx, fmt, hd, 2, G, [n], [1], seed=n + G)
    b.check(b.run())
    ctx.sync()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hd,H,G", [(64, 1, 5), (128, 2, 4), (128, 3, 7)])
@pytest.mark.parametrize("held,rows", [
    ([1, 700, 64, 128, 3], [1, 1, 1, 1, 1]),            # decode, ragged
    ([0, 5, 0, 65], [1, 1, 0, 1]),                      # nothing held, an unused slot of the batch
    ([5, 200, 1, 64], [5, 3, 1, 4]),                    # verify passes; all of a request's rows are all it holds
    ([2, 70, 4], [5, 8, 6]),                            # rows that see nothing
    ([300, 0, 129], [33, 0, 17]),                       # many rows
    ([0], [3]), ([64], [0, ]),
])
def test_batches(ctx, fmt, hd, H, G, held, rows):
    b = Batch(ctx, fmt, hd, H, G, held, rows, seed=sum(held) + hd)
    out = b.run(pad=2)
    if sum(rows):
        b.check(out)
    assert (host(out)[sum(rows):] == 123.0).all()       # rows of no request
    ctx.sync()


@pytest.mark.parametrize("n_req,n,rows", [(300, 40, 1), (64, 500, 2), (1024, 5, 1), (40, 900, 5)])
def test_many_requests(ctx, n_req, n, rows):
    rng = np.random.default_rng(n_req)
    held = [int(x) for x in rng.integers(0, n, n_req)]
    b = Batch(ctx, nt.KV4_I4, 64, 1, 2, held, [rows] * n_req, seed=1)
    b.check(b.run())
    ctx.sync()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,H,G,rows", [(70000, 1, 4, 1), (40000, 2, 8, 3), (9000, 8, 4, 1)])
def test_long(ctx, fmt, n, H, G, rows):
    b = Batch(ctx, fmt, 128, H, G, [n], [rows], seed=2)
    b.check(b.run())
    ctx.sync()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("width", [0, 192, 193, 5000])
@pytest.mark.parametrize("hd,H,G,held,rows", [
    (128, 2, 4, [520], [1]), (128, 1, 8, [12288], [1]), (64, 2, 4, [4160, 5, 0, 700], [1, 1, 1, 1]),
    (128, 4, 1, [12289, 64], [1, 1]), (64, 1, 2, [1536] * 5, [1] * 5), (128, 2, 8, [1025, 1], [2, 1]),
    (64, 3, 4, [512] * 32, [1] * 32), (64, 3, 4, [600] * 33, [1] * 33), (64, 8, 3, [9000] + [20] * 8, [1] * 9)])
def test_who_has_an_item(ctx, fmt, width, hd, H, G, held, rows):
    """Items of a CTA's own, of a cluster's own and in line, by the tables' width, the lengths and their number."""
    b = Batch(ctx, fmt, hd, H, G, held, rows, seed=len(held) + hd, width=width)
    b.check(b.run())
    ctx.sync()


@pytest.mark.parametrize("spread,q_size", [(4.0, 1e-3), (0.5, 60.0), (0.5, 1e-30), (0.0, 1e20)])
def test_sizes_of_q_and_values(ctx, spread, q_size):
    """Channels from 1e-7 to 1e5 apart in size; scores near zero, and so far apart that one position takes all."""
    if q_size == 1e20:
        b = Batch(ctx, nt.KV4_I4, 128, 1, 4, [500], [2], seed=3, q_size=q_size)
        want, _ = b.expect()
        got = host(b.run())
        # one position's value each, exact in f16, unless two scores tie within the bound
        near = np.abs(got - want) <= 2.0 ** -20 * np.abs(want).max()
        assert np.isfinite(got).all() and near.mean() > 0.9
        return
    b = Batch(ctx, nt.KV4_E2M1, 128, 2, 4, [500, 70], [2, 1], seed=3, spread=spread, q_size=q_size)
    b.check(b.run())


def test_values_of_very_unequal_size(ctx):
    """Pages whose V scales are at f16's ends."""
    b = Batch(ctx, nt.KV4_I4, 64, 1, 4, [320], [1], seed=4)
    for i, s in enumerate((2.0 ** -20, 3000.0, 1.0, 2.0 ** -17, 0.0)):
        b.v[0][64 * i:64 * i + 64] *= s
    p = np.arange(320)
    slots = host(b.table)[0, p // 64].astype(np.int64) * 64 + p % 64
    b.cache.append(dev(b.k[0]), dev(b.v[0]), dev(slots))
    b.check(b.run())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hd,H,G,held,rows", [(128, 2, 4, [300], [300]), (64, 1, 3, [1000, 7, 450], [1000, 7, 101]),
                                              (128, 1, 16, [130, 200], [130, 9])])
def test_prompts(ctx, fmt, hd, H, G, held, rows):
    """Prompts of many chunks of rows, from their first position on or behind others."""
    b = Batch(ctx, fmt, hd, H, G, held, rows, seed=15)
    b.check(b.run(pad=1))
    ctx.sync()


def test_nan_query_stays_in_its_row(ctx):
    b = Batch(ctx, nt.KV4_I4, 128, 2, 4, [300, 90], [1, 2], seed=5)
    want, bound = b.expect()
    b.q[1, 5, 7], b.q[0, 2, 3] = np.nan, np.inf
    got = host(b.run())
    bad = np.zeros(got.shape[:2], dtype=bool)
    bad[1, 5] = bad[0, 2] = True
    assert np.isnan(got[bad]).all()
    assert (np.abs(got - want)[~bad] <= bound[~bad]).all()


def test_output_in_place_and_repeated(ctx):
    """Bit-identical whatever runs before, and with the output in q's place."""
    b = Batch(ctx, nt.KV4_E2M1, 128, 8, 4, [3000, 70, 1500], [1, 4, 2], seed=6)
    first = host(b.run())
    for _ in range(5):
        q = dev(b.q)
        b.cache.attend(q, q, b.q_start, b.held_dev, b.table)
        assert np.array_equal(host(q), first)


def test_bad_pages_and_lengths(ctx):
    """What a table or a length has wrong is flagged and taken as absent; the rest is right."""
    b = Batch(ctx, nt.KV4_I4, 64, 2, 2, [200, 130, 100, 90], [1, 1, 1, 1], seed=7)
    table = host(b.table).copy()
    table[1, 1] = b.cache.n_pages            # its positions 64 .. 127 are not seen
    table[2, :] = -1                          # nothing is seen
    b.table = dev(table)
    b.held_dev = dev(np.array([200, 130, 100, -4], dtype=np.int32))
    got = host(b.run())
    with pytest.raises(nt.NtError, match="page"):
        ctx.sync()
    keep = np.r_[0:64, 128:130]
    parts = [(b.k[0], b.v[0]), (b.k[1][keep], b.v[1][keep])]
    for r, (k, v) in enumerate(parts):
        want, bound = ref.attend(b.q[r:r + 1], ref.values(k, 0), ref.values(v, 0), 1)
        assert (np.abs(got[r:r + 1] - want) <= bound).all()
    assert (got[2:] == 0).all()
    b.held_dev = dev(np.array([200, 64 * table.shape[1] + 1, 0, 90], dtype=np.int32))
    b.table = dev(np.where(table < 0, 0, np.minimum(table, b.cache.n_pages - 1)))
    b.run()
    with pytest.raises(nt.NtError, match="length"):
        ctx.sync()
    for q_start in ([0, 1, 3, 2, 4], [0, 1, 2, 3, 5], [-1, 1, 2, 3, 4]):
        b.q_start = dev(np.array(q_start, dtype=np.int32))
        b.held_dev = dev(np.array([200, 130, 0, 90], dtype=np.int32))
        got = host(b.run(pad=0))
        with pytest.raises(nt.NtError):
            ctx.sync()
    ctx.sync()


@pytest.mark.parametrize("n_req", [1, 40])
def test_more_work_than_the_call_takes(ctx, n_req):
    """More than 2^28 pages of heads to go through: flagged, and nothing is computed (or read: the table holds -1)."""
    cache = engine.KV4Cache(ctx, nt.KV4_I4, 64, 64, 1)
    pages = 2 ** 22 // n_req + 2 ** 16
    table = torch.full((n_req, pages), -1, dtype=torch.int32, device="cuda")
    held = torch.full((n_req,), 64 * pages, dtype=torch.int32, device="cuda")
    q_start = torch.arange(n_req + 1, dtype=torch.int32, device="cuda")
    q, out = torch.zeros(n_req, 64, 64, device="cuda"), torch.full((n_req, 64, 64), 7.0, device="cuda")
    cache.attend(q, out, q_start, held, table)
    with pytest.raises(nt.NtError, match="length"):
        ctx.sync()
    assert bool((out == 7.0).all())


def test_stale_pages_of_any_bytes(ctx):
    """Bytes behind a request's positions count for nothing, whatever they are."""
    for garbage in (0x00, 0x7C, 0x7F, 0xFC):                # huge and NaN scales among them
        for fmt in FMTS:
            b = Batch(ctx, fmt, 128, 2, 4, [65, 1, 127, 63], [2, 1, 3, 1], seed=9, garbage=garbage)
            b.check(b.run())
    ctx.sync()


def test_requests_that_share_pages(ctx):
    """Two requests with a common prefix read the same pages."""
    b = Batch(ctx, nt.KV4_E2M1, 128, 1, 4, [256, 100], [1, 1], seed=8)
    table = host(b.table).copy()
    table[1] = table[0]
    b.table = dev(table)
    b.k[1], b.v[1] = b.k[0][:100], b.v[0][:100]
    b.check(b.run())


def test_refusals(ctx):
    b = Batch(ctx, nt.KV4_I4, 64, 2, 2, [70], [1])
    q, out = dev(b.q), torch.full((1, 4, 64), 9.0, device="cuda")
    d = b.cache.desc

    def desc(**kw):
        c = nt.nt_kv4(d.fmt, d.n_kvh, d.head_dim, d.n_pages, d.data)
        for name, x in kw.items():
            setattr(c, name, x)
        return c

    def attend(cache=d, n_qh=4, n_tok=1, n_req=1, W=2, q=q, out=out, qs=b.q_start, held=b.held_dev, table=b.table):
        nt.nt_attn_kv4(ctx, q, cache, out, n_qh, n_tok, n_req, qs, held, table, W)

    k, s = torch.zeros(4, 2, 64, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")

    def rows(f, cache=d, fmt=nt.F32, k=k, v=k, n=4, ts=128, hs=64, s=s):
        f(ctx, cache, fmt, k, v, n, ts, hs, s)

    bad = [lambda: attend(cache=desc(fmt=2)), lambda: attend(cache=desc(head_dim=96)), lambda: attend(cache=desc(n_kvh=0)),
           lambda: attend(cache=desc(n_kvh=65)), lambda: attend(cache=desc(n_pages=0)), lambda: attend(cache=desc(n_pages=(1 << 26) + 1)),
           lambda: attend(cache=desc(data=None)), lambda: attend(cache=desc(data=d.data + 8)), lambda: attend(n_qh=3),
           lambda: attend(n_qh=34), lambda: attend(n_qh=0), lambda: attend(n_tok=-1), lambda: attend(n_tok=(1 << 24) + 1),
           lambda: attend(n_req=0), lambda: attend(n_req=1025), lambda: attend(W=0), lambda: attend(W=(1 << 24) + 1),
           lambda: attend(q=None), lambda: attend(out=None), lambda: attend(qs=None), lambda: attend(held=None),
           lambda: attend(table=None), lambda: attend(q=q.data_ptr() + 4), lambda: attend(out=out.data_ptr() + 4),
           lambda: attend(held=b.held_dev.data_ptr() + 2)]
    for f in (nt.nt_kv4_append, nt.nt_kv4_read):
        bad += [lambda f=f: rows(f, fmt=nt.Q8_0), lambda f=f: rows(f, n=-1), lambda f=f: rows(f, n=(1 << 28) + 1),
                lambda f=f: rows(f, ts=126), lambda f=f: rows(f, hs=66), lambda f=f: rows(f, k=k.data_ptr() + 8),
                lambda f=f: rows(f, fmt=nt.F16, hs=68), lambda f=f: rows(f, ts=1 << 41), lambda f=f: rows(f, s=s.data_ptr() + 4),
                lambda f=f: rows(f, cache=desc(fmt=-1))]
    bad += [lambda: rows(nt.nt_kv4_append, v=None), lambda: rows(nt.nt_kv4_read, k=None, v=None),
            lambda: rows(nt.nt_kv4_read, ts=64), lambda: rows(nt.nt_kv4_read, ts=0), lambda: rows(nt.nt_kv4_read, hs=-64),
            lambda: nt.nt_kv4_append(ctx, d, nt.F32, k, k, 4, 128, 64, None, stream=0),
            lambda: nt.nt_attn_kv4(ctx, q, None, out, 4, 1, 1, b.q_start, b.held_dev, b.table, 2)]
    for i, call in enumerate(bad):
        with pytest.raises(nt.NtError) as e:
            call()
        assert e.value.status in (nt.NT_ERR_INVALID_ARG, nt.NT_ERR_ALIGNMENT, nt.NT_ERR_UNSUPPORTED_FMT), i
    # nothing to do
    attend(n_tok=0, q=None, out=None)
    rows(nt.nt_kv4_append, n=0, k=None, v=None, s=s)
    rows(nt.nt_kv4_read, n=0)
    assert (host(out) == 9.0).all()
    ctx.sync()


def test_small_scratch(ctx):
    small = nt.Context(0, 1 << 20)
    b = Batch(small, nt.KV4_I4, 64, 1, 1, [70], [1])
    with pytest.raises(nt.NtError) as e:
        b.run()
    assert e.value.status == nt.NT_ERR_OOM
    small.close()


def test_copies_that_never_come(ctx):
    """A launch whose copies are left out reports the wait that ran out, and the next one is right."""
    b = Batch(ctx, nt.KV4_I4, 128, 8, 4, [3000, 200], [1, 1], seed=9)
    nt.nt_debug_stall_waits(1)
    b.run()
    with pytest.raises(nt.NtError) as e:
        ctx.sync()
    assert e.value.status == nt.NT_ERR_TIMEOUT
    nt.nt_debug_stall_waits(0)
    b.check(b.run())
    ctx.sync()


def test_contexts_on_two_streams(ctx):
    """Two contexts, each on a stream of its own, at the same time."""
    other = nt.Context(0)
    bs = [Batch(c, nt.KV4_I4, 128, 4, 4, [2000 + 64 * i, 90], [1, 3], seed=10 + i) for i, c in enumerate((ctx, other))]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in bs]
    qs = [dev(b.q) for b in bs]
    outs = [torch.empty_like(q) for q in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for b, s, q, o in zip(bs, streams, qs, outs):
            b.cache.attend(q, o, b.q_start, b.held_dev, b.table, stream=s)
    torch.cuda.synchronize()
    for b, o in zip(bs, outs):
        b.check(o)
    ctx.sync(), other.sync()
    other.close()


# ---- whole steps -----------------------------------------------------------------
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("captured", [False, True])
def test_steps_of_several_requests(ctx, fmt, captured):
    """Requests start with prompts, decode, verify drafts and drop some, end and start again: tables, rotated rows,
    cache writes and attention, run as a step's four calls (captured once and replayed, or not)."""
    R, W, n_pages, H, G, hd, cap = 4, 6, 17, 2, 4, 64, 40
    rng = np.random.default_rng(11)
    pages = engine.KV4Pages(ctx, R, W, n_pages)
    cache = engine.KV4Cache(ctx, fmt, H, hd, n_pages)
    rope = engine.Rope(ctx, hd, 48, nt.ROPE_HALVES, theta=10000.0, scaling=nt.ROPE_LINEAR, factor=4.0)
    freq = ref.frequencies(48, 10000.0, "linear", 4.0)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    new, keep, q_start, positions = i32(R), i32(R), i32(R + 1), i32(cap)
    slots = torch.zeros(cap, dtype=torch.int64, device="cuda")
    q, k, v = (torch.zeros(cap, n, hd, device="cuda") for n in (H * G, H, H))
    qr, kr, out = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(q)

    def step():
        pages.step(new, q_start, slots, positions, keep=keep)
        rope.rotate((q, qr), (k, kr), positions=positions)
        cache.append(kr, v, slots)
        cache.attend(qr, out, q_start, pages.held, pages.table)

    graph = None
    if captured:
        step()                       # no rows yet
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    # (keep, new) of each request in each step
    plan = [[(0, 30), (0, 1), (0, 0), (0, 5)], [(30, 1), (1, 1), (0, 33), (5, 5)], [(31, 1), (2, 1), (33, 1), (7, 5)],
            [(0, 0), (3, 1), (34, 31), (9, 5)], [(0, 20), (4, 0), (65, 1), (14, 1)], [(20, 1), (4, 1), (66, 1), (0, 0)]]
    hist = [[np.zeros((0, H, hd)), np.zeros((0, H, hd))] for _ in range(R)]
    for ks in plan:
        rows = [n for _, n in ks]
        total = sum(rows)
        data = [rng.standard_normal(t.shape).astype(np.float32) for t in (q, k, v)]
        for t, x in zip((q, k, v), data):
            t.copy_(torch.from_numpy(x))
        new.copy_(torch.tensor(rows, dtype=torch.int32))
        keep.copy_(torch.tensor([a for a, _ in ks], dtype=torch.int32))
        graph.replay() if captured else step()
        ctx.sync()
        got, at = host(out), 0
        assert host(pages.held).tolist() == [a + b for a, b in ks]
        assert host(slots)[total:].tolist() == [-1] * (cap - total)
        assert int(pages.n_free) == n_pages - sum(-(-(a + b) // 64) for a, b in ks)
        for r, (a, n) in enumerate(ks):
            pos = np.arange(a, a + n)
            assert host(positions)[at:at + n].tolist() == pos.tolist()
            # K is what the library's own rotation gave (fp32), so that the 4-bit codes are the same numbers
            assert np.abs(host(kr)[at:at + n] - ref.rotate(data[1][at:at + n], pos, freq, 1)).max(initial=0) < 1e-6
            hist[r] = [np.concatenate([old[:a], ref.values(x[at:at + n], fmt)]) for old, x in
                       zip(hist[r], (host(kr), data[2]))]
            want, bound = ref.attend(host(qr)[at:at + n].astype(np.float64), hist[r][0], hist[r][1], n)
            assert (np.abs(got[at:at + n] - want) <= bound).all()
            at += n


@pytest.mark.parametrize("fmt", FMTS)
def test_pages_past_2_to_32_bytes(ctx, fmt):
    """A pool of 4.4 GB: written, read back and attended at both of its ends."""
    rng = np.random.default_rng(13)
    n, H, hd, n_pages = 150, 8, 128, 60000
    data = torch.empty(n_pages, H, nt.nt_kv4_layout(hd), dtype=torch.uint8, device="cuda")
    cache = engine.KV4Cache(ctx, fmt, H, hd, n_pages, data=data)
    table = np.array([[59999, 0, 58300, -1]], dtype=np.int32)
    p = np.arange(n)
    slots = dev(table[0, p // 64].astype(np.int64) * 64 + p % 64)
    k, v = _rows(rng, n, H, hd), _rows(rng, n, H, hd)
    cache.append(dev(k), dev(v), slots)
    ko, vo = torch.empty(n, H, hd, device="cuda"), torch.empty(n, H, hd, device="cuda")
    cache.read(ko, vo, slots)
    kq, vq = ref.values(k, fmt), ref.values(v, fmt)
    assert np.array_equal(host(ko), kq.astype(np.float32)) and np.array_equal(host(vo), vq.astype(np.float32))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for rows in (1, 3):
        q = rng.standard_normal((rows, 4 * H, hd)).astype(np.float32)
        out = torch.empty(rows, 4 * H, hd, device="cuda")
        cache.attend(dev(q), out, i32(0, rows), i32(n), dev(table))
        want, bound = ref.attend(q, kq, vq, rows)
        assert (np.abs(host(out) - want) <= bound).all()
    ctx.sync()


def test_first_row_of_the_batch_is_not_the_first_request_s(ctx):
    """Rows before the first request's are left as they were, and slots read twice come twice."""
    b = Batch(ctx, nt.KV4_I4, 64, 2, 4, [70, 5], [2, 1], seed=14)
    q = np.concatenate([np.zeros((3,) + b.q.shape[1:], dtype=np.float32), b.q])
    out = torch.full(q.shape, 123.0, device="cuda")
    b.cache.attend(dev(q), out, b.q_start + 3, b.held_dev, b.table)
    assert (host(out)[:3] == 123.0).all()
    b.check(out[3:])
    slot = int(b.table[0, 1]) * 64 + 3
    ko, vo = torch.empty(3, 2, 64, device="cuda"), torch.empty(3, 2, 64, device="cuda")
    b.cache.read(ko, vo, torch.full((3,), slot, device="cuda"))
    for i in range(3):
        assert np.array_equal(host(ko)[i], ref.values(b.k[0], 0)[67].astype(np.float32))
    ctx.sync()


def test_memory_is_not_allocated(ctx):
    b = Batch(ctx, nt.KV4_I4, 128, 8, 4, [3000, 200], [1, 1], seed=12)
    q, out = dev(b.q), torch.empty(2, 32, 128, device="cuda")
    b.cache.attend(q, out, b.q_start, b.held_dev, b.table)
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    for _ in range(50):
        b.cache.attend(q, out, b.q_start, b.held_dev, b.table)
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free
