"""The 8-bit cache at the edges of its formats: blocks begun elsewhere with scales
that are no powers of two, the largest floats beside an infinity, V scales
from the least to nearly the largest, and what the sync reports of several causes."""
import math

import numpy as np
import pytest

import kv8_ref as ref
import kv8_tight as tight
from gpu_util import dev, host, need_gpu, torch

pytestmark = pytest.mark.gpu
I8, E4M3 = ref.I8, ref.E4M3


@pytest.fixture(scope="module")
def ctx():
    need_gpu()
    from block_quantized_gemv_nt_gb300 import nt
    c = nt.Context(0)
    yield c
    c.sync()
    c.close()


def _new(ctx, fmt, H, hd, n):
    from block_quantized_gemv_nt_gb300 import engine
    return engine.KV8Cache(ctx, fmt, H, hd, n), ref.Cache(fmt, H, hd, n)


def _upload(g, c):
    for w in "kv":
        g.buffers[w].copy_(torch.from_numpy(c.data[w]))
        g.buffers[w + "scale"].copy_(torch.from_numpy(c.scale[w].astype(np.float32)))


class Continued(ref.Cache):
    """A cache whose blocks may have been begun elsewhere: an old scale that is no power of two counts as the next one
    above it, and the block's earlier rows are rounded to the new scale (E4M3: from the fp32 product with the ratio)."""

    def _block(self, w, h, b, lo, hi, x):
        fmt, data, finite = self.fmt, self.data[w][h], np.abs(x)[np.isfinite(x)]
        t = ref.scale_for(finite.max() if finite.size else 0.0, ref.QMAX[fmt])
        if lo > b * ref.B:
            old = self.scale[w][h, b]
            t = max(t, old if math.frexp(old)[0] == 0.5 else 2.0 ** math.ceil(math.log2(old)))
            v = ref.to_values(data[b * ref.B:lo], fmt) * (old / t)
            # I8 -128 is a value of such a cache: it stays where the ratio rounds it
            q = np.rint(v) if fmt == I8 else ref.round8(v.astype(np.float32).astype(np.float64), fmt)
            data[b * ref.B:lo] = ref.to_bytes(q, fmt)
        data[lo:hi] = ref.to_bytes(ref.round8(np.where(np.isnan(x), 0.0, x) / t, fmt), fmt)
        self.scale[w][h, b] = t
        if w == "k":
            q, u = ref.to_values(data[b * ref.B:hi], fmt), 1.0 if fmt == I8 else 4.0
            self.kmin[h, b], self.kmax[h, b] = np.floor(q.min(axis=0) / u), np.ceil(q.max(axis=0) / u)


@pytest.mark.parametrize("src", ["f32", "f16"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("fmt", [I8, E4M3])
def test_append_continues_blocks_of_any_scale(ctx, fmt, hd, src):
    """Rows behind those of a cache quantised elsewhere: the old rows keep their values to half a step of the new
    scale, the new rows are right, in growing blocks and in blocks that need no larger scale."""
    H, n0, n1 = 3, 64 + 21, 64 * 2 + 9
    rng = np.random.default_rng(50 + fmt)
    g, _ = _new(ctx, fmt, H, hd, n1)
    for size in (0.01, 1.0, 300.0):
        c = Continued(fmt, H, hd, n1)
        for w in "kv":
            b = rng.integers(0, 256, size=(H, n1, hd), dtype=np.uint8)
            if fmt == E4M3:
                b[(b & 0x7F) == 0x7F] = 0x7E
            c.data[w] = b
            s = rng.uniform(0.01, 0.1, size=c.scale[w].shape).astype(np.float32)
            s[:, 0], s[0, 1], s[1, 1] = 0.03, 1.5 / 64, np.nextafter(np.float32(1 / 64), np.float32(0))
            c.scale[w] = s.astype(np.float64)
        c.data["k"][:, n0 - 1, 0] = 0x80 if fmt == I8 else 0xFE
        _upload(g, c)
        before = {w: c.read(w, np.arange(n0)) for w in "kv"}
        x = (rng.normal(size=(2, n1 - n0, H, hd)) * size).astype(np.float32 if src == "f32" else np.float16)
        at = n0
        for m in (1, 1, 45, n1 - n0 - 47):  # within the block, over its end
            rows = x[:, at - n0:at - n0 + m]
            g.append(dev(rows[0]), dev(rows[1]), at)
            c.append(rows[0], rows[1], at)
            at += m
            nb = ref.blocks(at)
            for w in "kv":
                assert np.array_equal(host(g.buffers[w + "scale"])[:, 1:nb].astype(np.float64), c.scale[w][:, 1:nb]), w
                assert np.array_equal(host(g.buffers[w])[:, :at], c.data[w][:, :at]), w
            assert np.array_equal(host(g.buffers["kmin"])[:, 1:nb], c.kmin[:, 1:nb])
            assert np.array_equal(host(g.buffers["kmax"])[:, 1:nb], c.kmax[:, 1:nb])
        ctx.sync()
        back = torch.empty(H, n1, hd, device="cuda"), torch.empty(H, n1, hd, device="cuda")
        g.read(0, *back)
        for w, got in zip("kv", back):
            got = host(got).astype(np.float64)
            t = host(g.buffers[w + "scale"]).astype(np.float64)[:, np.arange(n1) // 64][..., None]
            new = x["kv".index(w)].astype(np.float64).transpose(1, 0, 2)
            for have, want, step in ((got[:, 64:n0], before[w][:, 64:], t[:, 64:n0]), (got[:, n0:], new, t[:, n0:])):
                # half a step a rounding; the scale grows at most log2 times, each time by a factor of two or more
                half = step / 2 if fmt == I8 else np.maximum(np.abs(want) * 2.0 ** -4, step * 2.0 ** -10)
                assert np.all(np.abs(have - want) <= 2.0 * half * (1 + 2.0 ** -4)), w


@pytest.mark.parametrize("fmt", [I8, E4M3])
def test_infinity_beside_the_largest_floats(ctx, fmt):
    """An infinity is stored as the largest 8-bit value also in a block whose finite values reach the largest float,
    a NaN as 0; whole blocks and ragged ones."""
    from block_quantized_gemv_nt_gb300 import nt
    H, hd, n = 1, 64, 64 * 3 + 20
    g, c = _new(ctx, fmt, H, hd, n)
    top = np.finfo(np.float32).max
    rng = np.random.default_rng(51)
    x = (rng.uniform(-1, 1, size=(n, H, hd)) * top).astype(np.float32)
    x[70, 0, 3] = top
    x[64 * 3 + 2, 0, 3] = -top
    for r in (5, 71, 64 * 3 + 5):
        x[r, 0, 7], x[r, 0, 8], x[r, 0, 9] = np.inf, -np.inf, np.nan
    g.append(dev(x), dev(-x), 0)
    c.append(x, -x, 0)
    with pytest.raises(nt.NtError) as e:
        ctx.sync()
    assert e.value.status == nt.NT_ERR_INVALID_ARG
    for w in "kv":
        assert np.array_equal(host(g.buffers[w + "scale"]).astype(np.float64), c.scale[w]), w
        assert np.array_equal(host(g.buffers[w]), c.data[w]), w
    assert np.array_equal(host(g.buffers["kmin"]), c.kmin) and np.array_equal(host(g.buffers["kmax"]), c.kmax)


@pytest.mark.parametrize("fmt", [I8, E4M3])
@pytest.mark.parametrize("e", [-100, -90, -80, -66, -30, 0, 60, 90, 104, 112, 122])
def test_every_v_scale_is_accurate(ctx, fmt, e):
    """V scales of about 2^e throughout, e down to the least the append writes: the output is as accurate as at 1.
    One CTA a head, a cluster and two launches, one query and several."""
    from block_quantized_gemv_nt_gb300 import nt  # noqa: F401
    H, G, hd = 2, 4, 128
    rng = np.random.default_rng(e + 200)
    for n, nq in ((150, 1), (1500, 1), (20001, 1), (1500, 7)):
        g, c = _new(ctx, fmt, H, hd, n + nq - 1)
        for w in "kv":
            size = 1 if w == "v" and e > 112 else 30  # (the values stay below the largest float)
            b = np.clip(np.rint(rng.normal(size=c.data[w].shape) * size), -127, 127)
            c.data[w] = b.astype(np.int8).view(np.uint8) if fmt == I8 else ref.to_bytes(ref.round8(b, fmt), fmt)
        c.scale["k"][:] = 2.0 ** -5
        up = rng.integers(0, 3, size=c.scale["v"].shape)
        c.scale["v"] = 2.0 ** (e + up if e < 100 else e - up)
        _upload(g, c)
        q = rng.normal(size=(nq, H * G, hd)).astype(np.float32)
        out = torch.empty((nq, H * G, hd), device="cuda")
        g.attend(dev(q), out, n)
        ctx.sync()
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        tight.check(host(out), c, q, n, tight.plan(sms, H, G, hd, nq, n))


@pytest.mark.parametrize("fmt", [I8, E4M3])
def test_written_tiny_values_are_attended_to(ctx, fmt):
    """Rows of v around 1e-28 through the append: their scales lie near the least, and the attention over them, over
    blocks of 1 among them and over all-zero blocks keeps its accuracy."""
    H, G, hd, n = 1, 4, 64, 64 * 6
    rng = np.random.default_rng(52)
    g, c = _new(ctx, fmt, H, hd, n)
    k, v = (rng.normal(size=(n, H, hd)).astype(np.float32) for _ in range(2))
    v[:] *= np.float32(1e-28)
    v[64:128] = 0
    g.append(dev(k), dev(v), 0)
    c.append(k, v, 0)
    q = rng.normal(size=(1, G, hd)).astype(np.float32)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    out = torch.empty((1, G, hd), device="cuda")
    for n_pos in (64, 200, n):
        g.attend(dev(q), out, n_pos)
        tight.check(host(out), c, q, n_pos, tight.plan(sms, H, G, hd, 1, n_pos))
    for size in (1.0, 1e9, 1e30):
        v[256:320] = rng.normal(size=(64, H, hd)) * size
        g.append(dev(k), dev(v), 0)
        c.append(k, v, 0)
        g.attend(dev(q), out, n)
        tight.check(host(out), c, q, n, tight.plan(sms, H, G, hd, 1, n), rms=False)
    ctx.sync()


@pytest.mark.parametrize("order", ["large first", "large last"])
@pytest.mark.parametrize("fmt", [I8, E4M3])
def test_zero_blocks_keep_their_weight(ctx, fmt, order):
    """One warp walks a block of large values and then all-zero ones, or the other way round: the zeros' probabilities
    stay in the sum, however large the other block is."""
    H, G, hd, blocks = 1, 4, 64, 76 * 8
    rng = np.random.default_rng(53)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    g, c = _new(ctx, fmt, H, hd, 64 * blocks)
    for w in "kv":
        b = np.clip(np.rint(rng.normal(size=c.data[w].shape) * 30), -127, 127)
        c.data[w] = b.astype(np.int8).view(np.uint8) if fmt == I8 else ref.to_bytes(ref.round8(b, fmt), fmt)
    c.scale["k"][:] = 2.0 ** -5
    q = rng.normal(size=(1, G, hd)).astype(np.float32)
    out = torch.empty((1, G, hd), device="cuda")
    p = tight.plan(sms, H, G, hd, 1, 64 * blocks)
    for e in (0, 30, 60, 100):
        zero = np.ones(blocks, bool)
        zero[slice(0, blocks // 4) if order == "large first" else slice(blocks - blocks // 4, blocks)] = False
        c.scale["v"][:] = np.where(zero, 2.0 ** -100, 2.0 ** e)
        c.data["v"][:, np.repeat(zero, 64)] = 0
        _upload(g, c)
        g.attend(dev(q), out, 64 * blocks)
        tight.check(host(out), c, q, 64 * blocks, p)
    # one CTA, lists of one large block among zeros: every warp meets both
    at = np.flatnonzero(~zero)[:4]
    n_sel = 40
    lists = np.concatenate([np.flatnonzero(zero)[:n_sel // 2], at, np.flatnonzero(zero)[n_sel // 2:n_sel - 4]])
    lists = lists[None, None] if order == "large last" else lists[None, None, ::-1]
    g.attend_blocks(dev(q), out, 64 * blocks, dev(np.ascontiguousarray(lists).astype(np.int32)))
    tight.check(host(out), c, q, 64 * blocks, tight.plan(sms, H, G, hd, 1, 64 * blocks, n_sel), lists)
    ctx.sync()


@pytest.mark.parametrize("fmt", [I8, E4M3])
@pytest.mark.parametrize("span", [(-100, 122), (-100, 60), (-45, 100), (0, 122)])
def test_v_scales_in_any_mix(ctx, fmt, span):
    """Blocks of V scales all over the range, every position about as probable: each block's probabilities count in the
    sum, and the outputs are those of the largest.  In every order a warp or a merge can meet them."""
    H, G, hd = 1, 4, 64
    rng = np.random.default_rng(55)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for n in (150, 700, 5000, 64 * 76 * 8):
        g, c = _new(ctx, fmt, H, hd, n)
        for w in "kv":
            b = np.clip(np.rint(rng.normal(size=c.data[w].shape) * (20 if w == "k" else 1)), -127, 127)
            c.data[w] = b.astype(np.int8).view(np.uint8) if fmt == I8 else ref.to_bytes(ref.round8(b, fmt), fmt)
        c.scale["k"][:] = 2.0 ** -5
        q = rng.normal(size=(1, G, hd)).astype(np.float32)
        out = torch.empty((1, G, hd), device="cuda")
        nb = c.scale["v"].shape[1]
        few = np.where(rng.random(nb) < 0.1, span[1], span[0])  # mostly the least, some the largest
        for e in (rng.integers(span[0], span[1] + 1, size=nb), few, np.sort(few), np.sort(few)[::-1]):
            c.scale["v"][0] = 2.0 ** e.astype(np.float64)
            _upload(g, c)
            g.attend(dev(q), out, n)
            tight.check(host(out), c, q, n, tight.plan(sms, H, G, hd, 1, n), rms=False)
    ctx.sync()


@pytest.mark.parametrize("fmt", [I8, E4M3])
@pytest.mark.parametrize("s", [-700.0, -90.0, 90.0, 700.0])
def test_scores_far_from_zero(ctx, fmt, s):
    """Every score about s, far below or above zero, with ordinary and with all-zero V blocks, from one position on."""
    H, G, hd = 1, 4, 64
    rng = np.random.default_rng(54)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for n in (1, 70, 1500, 40000):
        g, c = _new(ctx, fmt, H, hd, n)
        for w in "kv":
            b = np.rint(rng.normal(size=c.data[w].shape) * 10).clip(-40, 40) + (64 if w == "k" else 0)
            c.data[w] = b.astype(np.int8).view(np.uint8) if fmt == I8 else ref.to_bytes(ref.round8(b, fmt), fmt)
        c.scale["k"][:] = 2.0 ** -6
        c.scale["v"][:] = 2.0 ** -5
        if n > 64:
            c.data["v"][:, :64], c.scale["v"][:, 0] = 0, 2.0 ** -100
        _upload(g, c)
        q = (s / 8 + 0.2 * rng.normal(size=(1, G, hd))).astype(np.float32)  # s = 64 (s / 8) 1 / 8
        out = torch.empty((1, G, hd), device="cuda")
        g.attend(dev(q), out, n)
        tight.check(host(out), c, q, n, tight.plan(sms, H, G, hd, 1, n), rms=False)
    ctx.sync()


def test_sync_names_every_cause(ctx):
    """A row that is not finite and a device position past the end between two syncs: the report names both."""
    from block_quantized_gemv_nt_gb300 import nt
    g, _ = _new(ctx, I8, 1, 64, 100)
    x = torch.zeros(1, 1, 64, device="cuda")
    x[0, 0, 3] = float("nan")
    pos = torch.tensor([100], dtype=torch.int64, device="cuda")

    def report():
        with pytest.raises(nt.NtError) as e:
            ctx.sync()
        return e.value.status, str(e.value)

    g.append(x, x, 5)
    g.append(x, x, 0, pos_dev=pos)
    status, text = report()
    assert status == nt.NT_ERR_INVALID_ARG and "infinity" in text and "position" in text
    q = torch.ones(1, 1, 64, device="cuda")
    g.append(x, x, 5)
    nt.nt_debug_stall_waits(1)
    try:
        g.attend(q, torch.empty_like(q), 6)
    finally:
        nt.nt_debug_stall_waits(0)
    status, text = report()
    assert status == nt.NT_ERR_TIMEOUT and "infinity" in text and "position" not in text
    g.append(x, x, 5)
    status, text = report()
    assert status == nt.NT_ERR_INVALID_ARG and "infinity" in text and "position" not in text
    ctx.sync()
