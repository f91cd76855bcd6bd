"""The 8-bit KV cache on the GPU against the 64-bit numpy oracle (kv8_ref):
rows quantised as they are written and read back (bit-exact), attention over
the cache, block selection (exact indices) and attention over chosen blocks."""
import numpy as np
import pytest

import kv8_ref as ref
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


def _mods():
    from block_quantized_gemv_nt_gb300 import engine, nt
    return engine, nt


def _cache(ctx, fmt, H, hd, stride):
    """A device cache and its oracle; the device buffers start as noise (nothing needs initialising)."""
    engine, _ = _mods()
    g = engine.KV8Cache(ctx, fmt, H, hd, stride)
    gen = torch.Generator(device="cuda").manual_seed(7)
    for n in ("k", "v"):
        g.buffers[n].random_(0, 256, generator=gen)
    for n in ("kmin", "kmax"):
        g.buffers[n].random_(-128, 128, generator=gen)
    for n in ("kscale", "vscale"):
        g.buffers[n].fill_(float("nan"))
    return g, ref.Cache(fmt, H, hd, stride)


def _rows(rng, n, H, hd, grow=0.0):
    size = np.exp(0.5 * rng.normal(size=(1, H, hd))) * np.exp(grow * np.arange(n) / max(n, 1))[:, None, None]
    return (rng.normal(size=(n, H, hd)) * size).astype(np.float32)


def _same(g, c, n):
    """The device state equals the oracle's for positions below n."""
    nb = ref.blocks(n)
    for w in "kv":
        assert np.array_equal(host(g.buffers[w])[:, :n], c.data[w][:, :n]), w
        assert np.array_equal(host(g.buffers[w + "scale"])[:, :nb].astype(np.float64), c.scale[w][:, :nb]), w
    assert np.array_equal(host(g.buffers["kmin"])[:, :nb], c.kmin[:, :nb])
    assert np.array_equal(host(g.buffers["kmax"])[:, :nb], c.kmax[:, :nb])


# ---- refusals (all before any launch) ----------------------------------------------
def test_refusals(ctx):
    engine, nt = _mods()
    g = engine.KV8Cache(ctx, I8, 2, 128, 100)
    f = torch.zeros(4096, device="cuda")
    i = torch.full((64,), -7, dtype=torch.int32, device="cuda")

    def refuse(status, call):
        with pytest.raises(nt.NtError) as e:
            call()
        assert e.value.status == status and len(str(e.value)) > 10

    def desc(**kw):
        d = nt.nt_kv8.from_buffer_copy(g.desc)
        for k, v in kw.items():
            setattr(d, k, v)
        return d

    bad, fmt, align, oom = nt.NT_ERR_INVALID_ARG, nt.NT_ERR_UNSUPPORTED_FMT, nt.NT_ERR_ALIGNMENT, nt.NT_ERR_OOM
    app = lambda d=g.desc, src=nt.F32, k=f, v=f, n=1, ts=256, hs=128, pos=0, pd=None: (  # noqa: E731
        nt.nt_kv8_append(ctx, d, src, k, v, n, ts, hs, pos, pd, stream=0))
    for d, st in [(desc(fmt=2), fmt), (desc(head_dim=96), bad), (desc(n_kvh=0), bad), (desc(n_kvh=65), bad),
                  (desc(kv_stride=0), bad), (desc(kv_stride=2 ** 30 + 1), bad), (desc(k=None), bad),
                  (desc(vscale=None), bad), (desc(kmin=None), bad), (desc(v=g.desc.v + 8), align),
                  (desc(kscale=g.desc.kscale + 2), align), (desc(kmax=g.desc.kmax + 4), align)]:
        refuse(st, lambda: app(d))
        refuse(st, lambda: nt.nt_kv8_read(ctx, d, 0, 1, nt.F32, f, f, 128))
        refuse(st, lambda: nt.nt_attn_kv8(ctx, f, d, f, 4, 1))
        refuse(st, lambda: nt.nt_attn_kv8_blocks(ctx, f, d, f, 4, 1, 1, i, 4))
        refuse(st, lambda: nt.nt_kv8_select(ctx, f, d, 4, 1, 1, 4, 0, 1, i))
    p = f.data_ptr()
    refuse(fmt, lambda: app(src=nt.Q8_0))
    for kw in [dict(n=-1), dict(n=101), dict(pos=-1), dict(pos=100), dict(n=2, pos=99), dict(k=None), dict(v=None)]:
        refuse(bad, lambda: app(**kw))
    for kw in [dict(k=p + 8), dict(v=p + 4), dict(ts=130), dict(hs=2), dict(pd=p + 4), dict(src=nt.F16, k=p + 8),
               dict(src=nt.F16, ts=260), dict(src=nt.F16, hs=132)]:
        refuse(align, lambda: app(**kw))
    rd = lambda pos=0, n=1, t=nt.F32, k=f, v=f, hs=128: nt.nt_kv8_read(ctx, g.desc, pos, n, t, k, v, hs, stream=0)  # noqa: E731
    refuse(fmt, lambda: rd(t=nt.Q4_0))
    for kw in [dict(pos=-1), dict(pos=101), dict(n=-1), dict(pos=99, n=2), dict(k=None, v=None), dict(n=2)]:
        refuse(bad, lambda: rd(**kw))
    for kw in [dict(k=p + 4), dict(hs=130), dict(t=nt.F16, hs=132)]:
        refuse(align, lambda: rd(**kw))
    att = lambda q=f, o=f, H=4, n=1, nq=1, pd=None: nt.nt_attn_kv8(ctx, q, g.desc, o, H, n, nq, pd, stream=0)  # noqa: E731
    sel = lambda q=f, H=4, n=1, nq=1, ns=4, a=0, b=1, x=i, d=g.desc, pd=None: (  # noqa: E731
        nt.nt_kv8_select(ctx, q, d, H, n, nq, ns, a, b, x, pd, stream=0))
    blk = lambda q=f, o=f, H=4, n=1, nq=1, x=i, ns=4, pd=None: (  # noqa: E731
        nt.nt_attn_kv8_blocks(ctx, q, g.desc, o, H, n, nq, x, ns, pd, stream=0))
    for call in (att, sel, blk):
        for kw in [dict(q=None), dict(H=0), dict(H=3), dict(H=34), dict(n=-1), dict(n=101), dict(n=100, nq=2),
                   dict(nq=0), dict(nq=17)]:
            refuse(bad, lambda: call(**kw))
        for kw in [dict(q=p + 4), dict(pd=p + 4)]:
            refuse(align, lambda: call(**kw))
    for call in (att, blk):
        refuse(bad, lambda: call(o=None))
        refuse(align, lambda: call(o=p + 8))
    for call in (sel, blk):
        for kw in [dict(x=None), dict(ns=0), dict(ns=2 ** 24 + 1)]:
            refuse(bad, lambda: call(**kw))
        refuse(align, lambda: call(x=i.data_ptr() + 2))
    for kw in [dict(a=-1), dict(b=-1), dict(a=5, b=0), dict(a=3, b=2), dict(d=desc(kmin=None, kmax=None))]:
        refuse(bad, lambda: sel(**kw))
    small = nt.Context(0, 1 << 20)
    try:
        with pytest.raises(nt.NtError) as e:
            nt.nt_attn_kv8(small, f, g.desc, f, 4, 1)
        assert e.value.status == oom
        with pytest.raises(nt.NtError) as e:  # 2^22 blocks: their keys go to scratch
            nt.nt_kv8_select(small, f, desc(kv_stride=2 ** 28), 4, 2 ** 28, 1, 4, 0, 1, i)
        assert e.value.status == oom
    finally:
        small.close()
    app(n=0)  # nothing to do is no error
    rd(n=0)
    torch.cuda.synchronize()
    assert not f.any() and bool((i == -7).all())


# ---- write and read back --------------------------------------------------------------
@pytest.mark.parametrize("fmt", [I8, E4M3])
@pytest.mark.parametrize("H,hd,pieces", [(1, 128, [(0, 1)]), (3, 64, [(0, 63), (63, 1), (64, 1)]),
                                         (8, 128, [(0, 64), (64, 65), (129, 200)]), (2, 128, [(0, 333), (333, 5)]),
                                         (5, 64, [(0, 7), (7, 120), (127, 2)])])
def test_write_then_read(ctx, fmt, H, hd, pieces):
    rng = np.random.default_rng(100 * H + hd + fmt)
    end = pieces[-1][0] + pieces[-1][1]
    g, c = _cache(ctx, fmt, H, hd, end + 3)
    before = {w: host(g.buffers[w])[:, end:].copy() for w in "kv"}
    for j, (pos, n) in enumerate(pieces):
        k, v = _rows(rng, n, H, hd, 1.0) * 4.0 ** j, _rows(rng, n, H, hd)
        g.append(dev(k), dev(v), pos)
        c.append(k, v, pos)
        _same(g, c, pos + n)
    for w in "kv":  # rows behind the last one are left as they were
        assert np.array_equal(host(g.buffers[w])[:, end:], before[w])
    for pos, n in [(0, end), (end - 1, 1), (min(5, end - 1), end - min(5, end - 1))]:
        want = {w: c.read(w, np.arange(pos, pos + n)) for w in "kv"}
        for dt, npdt in ((torch.float32, np.float32), (torch.float16, np.float16)):
            k = torch.full((H, n, hd), 9.0, dtype=dt, device="cuda")
            v = torch.full((H, n + 1, hd), 9.0, dtype=dt, device="cuda")[:, :n]  # heads further apart
            k2 = torch.empty_strided(v.shape, v.stride(), dtype=dt, device="cuda")
            g.read(pos, k2, v)
            _, nt = _mods()
            nt.nt_kv8_read(ctx, g.desc, pos, n, nt.F32 if dt == torch.float32 else nt.F16, k, None, n * hd)
            assert np.array_equal(host(v), want["v"].astype(npdt)) and np.array_equal(host(k), want["k"].astype(npdt))
            assert np.array_equal(host(k2), host(k))


@pytest.mark.parametrize("fmt", [I8, E4M3])
def test_token_by_token_with_growth_and_rollback(ctx, fmt):
    """One token at a time with growing values (scales grow inside blocks), cut back twice across a block's end."""
    rng = np.random.default_rng(11)
    H, hd = 2, 128
    g, c = _cache(ctx, fmt, H, hd, 200)
    k, v = _rows(rng, 400, H, hd, 7.0), _rows(rng, 400, H, hd, -3.0)
    t = 0
    for start, stop in [(0, 70), (61, 140), (127, 150)]:
        for pos in range(start, stop):
            g.append(dev(k[t:t + 1]), dev(v[t:t + 1]), pos)
            c.append(k[t:t + 1], v[t:t + 1], pos)
            t += 1
        _same(g, c, stop)


def test_write_strides_and_f16_cache(ctx):
    """Rows of another layout: f16, heads first (an F16 cache), padded strides, one row repeated (stride 0)."""
    rng = np.random.default_rng(12)
    H, hd, n = 3, 64, 130
    x16 = _rows(rng, 150, H, hd).astype(np.float16)
    g, c = _cache(ctx, I8, H, hd, 140)
    heads = dev(np.ascontiguousarray(x16.transpose(1, 0, 2)))
    g.append_from_heads(heads[:, 10:10 + n], heads[:, 20:20 + n], 5)
    c.append(x16[10:10 + n], x16[20:20 + n], 5)
    nb = ref.blocks(5 + n)
    for w in "kv":
        assert np.array_equal(host(g.buffers[w])[:, 5:5 + n], c.data[w][:, 5:5 + n])
        assert np.array_equal(host(g.buffers[w + "scale"])[:, 1:nb], c.scale[w][:, 1:nb])
    g, c = _cache(ctx, E4M3, H, hd, 140)
    wide = dev(np.zeros((n, H + 2, hd + 4), np.float32))
    x = _rows(rng, n, H, hd)
    wide[:, 1:1 + H, :hd] = dev(x)
    view = torch.as_strided(wide, (n, H, hd), ((H + 2) * (hd + 4), hd + 4, 1), hd + 4)
    g.append(view, view, 0)
    c.append(x, x, 0)
    _same(g, c, n)
    g, c = _cache(ctx, E4M3, H, hd, 140)
    g.append(dev(x[:1]).expand(70, H, hd), dev(x[:1]).expand(70, H, hd), 0)
    c.append(np.repeat(x[:1], 70, 0), np.repeat(x[:1], 70, 0), 0)
    _same(g, c, 70)


@pytest.mark.parametrize("fmt", [I8, E4M3])
@pytest.mark.parametrize("hd", [64, 128])
def test_write_f16_rows(ctx, fmt, hd):
    """F16 rows, whole blocks and ragged ones: every f16 magnitude from subnormals to 65504, ties, a block with an
    infinity, one with a NaN, and blocks so small that 1 / scale is no f16 number."""
    _, nt = _mods()
    rng = np.random.default_rng(40 + fmt)
    H, n = 2, 64 * 12 + 30
    x = rng.normal(size=(n, H, hd)) * np.exp2(rng.integers(-3, 4, size=(n, H, 1)))
    x *= np.repeat(np.exp2(np.array([0, -24, -20, -14, -9, -8, -6, 3, 10, 13, 0, 0, 0.0])), 64)[:n, None, None]
    x[64 * 10:64 * 11] = (np.arange(64) - 31.5)[:, None, None] / 2
    x = np.clip(x, -65504, 65504).astype(np.float16)
    x[0, 0, 0], x[64 * 9, 0, 3], x[64 * 9 + 1, 1, 4] = 65504, 65504, -65504
    g, c = _cache(ctx, fmt, H, hd, n + 10)
    d = dev(x)
    g.append(d[:100], d[:100], 0)
    g.append(d[100:], d[100:], 100)
    c.append(x[:100], x[:100], 0)
    c.append(x[100:], x[100:], 100)
    ctx.sync()
    _same(g, c, n)
    y = x[:128].copy()
    y[70, 0, 5], y[71, 1, 6], y[72, 1, 7] = np.nan, np.inf, -np.inf
    g.append(dev(y), dev(y), 0)
    c.append(y, y, 0)
    with pytest.raises(nt.NtError):
        ctx.sync()
    nb = ref.blocks(128)
    for w in "kv":
        assert np.array_equal(host(g.buffers[w])[:, :128], c.data[w][:, :128])
        assert np.array_equal(host(g.buffers[w + "scale"])[:, :nb].astype(np.float64), c.scale[w][:, :nb])
    assert np.array_equal(host(g.buffers["kmin"])[:, :nb], c.kmin[:, :nb])
    assert np.array_equal(host(g.buffers["kmax"])[:, :nb], c.kmax[:, :nb])


@pytest.mark.parametrize("fmt", [I8, E4M3])
def test_write_extremes_and_non_finite(ctx, fmt):
    """Zeros, the smallest and largest floats, values at a scale's border; NaN and infinities are stored as 0
    and as the largest value, move no scale, and are reported by the sync."""
    _, nt = _mods()
    H, hd = 1, 64
    g, c = _cache(ctx, fmt, H, hd, 64 * 8)
    q = ref.QMAX[fmt]
    x = np.zeros((64 * 8, H, hd), np.float32)
    x[64] = 1e-45
    x[128:192] = 2.0 ** 126
    x[192, 0, 0], x[256, 0, 0] = q, np.nextafter(np.float32(q), np.float32(1e9))
    x[320:384, 0, :] = (np.arange(64) - 31.5)[None] / 2
    x[384:448, 0, :] = 127.0 * 2.0 ** -100
    x[448] = -0.0
    g.append(dev(x), dev(-x), 0)
    c.append(x, -x, 0)
    ctx.sync()
    for w in "kv":
        assert np.array_equal(host(g.buffers[w + "scale"]).astype(np.float64), c.scale[w])
    at = np.arange(64 * 8)
    k = torch.empty(H, 64 * 8, hd, device="cuda")
    g.read(0, k, torch.empty_like(k))
    assert np.array_equal(host(k), c.read("k", at).astype(np.float32))
    y = _rows(np.random.default_rng(13), 64, H, hd)
    y[3, 0, 5], y[4, 0, 6], y[5, 0, 7] = np.nan, np.inf, -np.inf
    g.append(dev(y), dev(y), 0)
    c.append(y, y, 0)
    with pytest.raises(nt.NtError) as e:
        ctx.sync()
    assert e.value.status == nt.NT_ERR_INVALID_ARG and "infinity" in str(e.value)
    ctx.sync()  # reported once
    _same(g, c, 64)


# ---- attention ---------------------------------------------------------------------------
def _filled(ctx, fmt, H, hd, n, stride, seed, poison=True):
    rng = np.random.default_rng(seed)
    g, c = _cache(ctx, fmt, H, hd, stride)
    k, v = _rows(rng, n, H, hd), _rows(rng, n, H, hd)
    if n:
        g.append(dev(k), dev(v), 0)
        c.append(k, v, 0)
    if poison and n < stride:  # rows nobody sees: bytes that are NaN in E4M3, scales that are NaN
        for w in "kv":
            g.buffers[w][:, n:] = 0x7F
            g.buffers[w + "scale"][:, ref.blocks(n):] = float("nan")
    return g, c, rng


def _check(got, want, tol):
    err = np.abs(got.astype(np.float64) - want)
    assert np.all(err <= tol), (np.max(err / tol), np.max(err))


LENGTHS = [(0, 1), (1, 1), (15, 1), (16, 3), (17, 1), (63, 2), (64, 1), (65, 16), (200, 5), (1088, 1), (4161, 8)]


@pytest.mark.parametrize("fmt", [I8, E4M3])
@pytest.mark.parametrize("n_pos,nq", LENGTHS)
def test_attention_lengths(ctx, fmt, n_pos, nq):
    H, G, hd = 2, 4, 128
    n = n_pos + nq - 1
    g, c, rng = _filled(ctx, fmt, H, hd, n, n + 70, 100 + n_pos)
    q = (rng.normal(size=(nq, H * G, hd)) * 1.5).astype(np.float32)
    out = torch.full((nq, H * G, hd), 5.0, device="cuda")
    g.attend(dev(q), out, n_pos)
    want, tol = ref.attend_cache(c, q, n_pos)
    _check(host(out), want, tol)
    if n_pos == 0:
        assert not host(out)[0].any()
    ctx.sync()


@pytest.mark.parametrize("fmt", [I8, E4M3])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("H,G,nq", [(1, 1, 1), (8, 1, 2), (3, 3, 1), (4, 7, 1), (8, 8, 1), (2, 16, 1), (2, 16, 16),
                                    (1, 5, 7), (64, 2, 1), (2, 3, 6), (1, 11, 3), (3, 16, 2), (1, 1, 16)])
def test_attention_heads(ctx, fmt, hd, H, G, nq):
    n_pos = 777
    g, c, rng = _filled(ctx, fmt, H, hd, n_pos + nq - 1, n_pos + nq - 1, 200 + H)
    q = (rng.normal(size=(nq, H * G, hd)) * 1.5).astype(np.float32)
    out = torch.empty((nq, H * G, hd), device="cuda")
    g.attend(dev(q), out, n_pos)
    _check(host(out), *ref.attend_cache(c, q, n_pos))


@pytest.mark.parametrize("fmt", [I8, E4M3])
def test_attention_long_and_peaky(ctx, fmt):
    """20,001 positions over every split; scores large enough that a few positions carry the sum."""
    H, G, hd, n_pos = 2, 4, 128, 20001
    g, c, rng = _filled(ctx, fmt, H, hd, n_pos, n_pos + 1, 300)
    for size in (1.0, 40.0):
        q = (rng.normal(size=(1, H * G, hd)) * size).astype(np.float32)
        out = torch.empty((1, H * G, hd), device="cuda")
        g.attend(dev(q), out, n_pos)
        want, tol = ref.attend_cache(c, q, n_pos)
        _check(host(out), want, tol)
        again = torch.empty_like(out)
        g.attend(dev(q), again, n_pos)
        assert torch.equal(out, again)


def test_attention_scale_ranges(ctx):
    """Blocks whose V (or K) scales lie far apart, an all-zero block, rows of q of very different size."""
    H, G, hd, n = 1, 4, 128, 64 * 5
    rng = np.random.default_rng(14)
    for fmt in (I8, E4M3):
        g, c = _cache(ctx, fmt, H, hd, n)
        k, v = _rows(rng, n, H, hd), _rows(rng, n, H, hd)
        k[64:128] = 0
        v[64:128] *= 1e-12
        v[128:192] = 0
        v[192:256] *= 1e9
        g.append(dev(k), dev(v), 0)
        c.append(k, v, 0)
        q = (rng.normal(size=(1, G, hd)) * np.array([1e-30, 1.0, 20.0, 0.0])[None, :, None]).astype(np.float32)
        out = torch.empty((1, G, hd), device="cuda")
        for n_pos in (64, 128, 192, n):
            g.attend(dev(q), out, n_pos)
            _check(host(out), *ref.attend_cache(c, q, n_pos))


@pytest.mark.parametrize("fmt", [I8, E4M3])
def test_attention_any_scales(ctx, fmt):
    """Scales that are no powers of two (a cache quantised elsewhere), every byte of I8 (-128 included)."""
    H, G, hd, n = 2, 4, 128, 64 * 9 + 5
    g, c, rng = _filled(ctx, fmt, H, hd, n, n, 28)
    for w in "kv":
        c.scale[w] = (c.scale[w] * rng.uniform(0.3, 3.0, size=c.scale[w].shape)).astype(np.float32).astype(np.float64)
        g.buffers[w + "scale"].copy_(torch.from_numpy(c.scale[w].astype(np.float32)))
        if fmt == I8:
            c.data[w][:, :32] = rng.integers(0, 256, size=c.data[w][:, :32].shape, dtype=np.uint8)
            c.data[w][:, 3] = 0x80
            g.buffers[w].copy_(torch.from_numpy(c.data[w]))
    for nq in (1, 5):
        q = rng.normal(size=(nq, H * G, hd)).astype(np.float32)
        out = torch.empty((nq, H * G, hd), device="cuda")
        g.attend(dev(q), out, n - nq + 1)
        _check(host(out), *ref.attend_cache(c, q, n - nq + 1))


def test_attention_nan_query_stays_in_its_row(ctx):
    H, G, hd, n = 2, 4, 128, 300
    g, c, rng = _filled(ctx, I8, H, hd, n, n, 15)
    q = rng.normal(size=(1, H * G, hd)).astype(np.float32)
    clean = torch.empty((1, H * G, hd), device="cuda")
    g.attend(dev(q), clean, n)
    q[0, 3, 17] = np.nan
    out = torch.empty_like(clean)
    g.attend(dev(q), out, n)
    a, b = host(out)[0], host(clean)[0]
    assert np.all(np.isnan(a[3])) and np.array_equal(np.delete(a, 3, 0), np.delete(b, 3, 0))


# ---- selection and sparse attention --------------------------------------------------------
@pytest.mark.parametrize("fmt", [I8, E4M3])
@pytest.mark.parametrize("H,G,hd,n_pos,nq,n_sel,first,last", [
    (2, 4, 128, 1, 1, 3, 0, 1), (2, 4, 128, 64 * 5, 1, 5, 1, 1), (2, 4, 128, 64 * 5, 2, 5, 1, 1),
    (8, 4, 128, 4160, 1, 16, 1, 2), (3, 7, 64, 5003, 5, 9, 0, 0), (1, 16, 64, 130, 1, 1, 0, 1),
    (2, 1, 128, 20001, 1, 100, 2, 4), (1, 2, 64, 70000, 1, 1050, 0, 3), (1, 2, 128, 0, 1, 4, 1, 1)])
def test_select(ctx, fmt, H, G, hd, n_pos, nq, n_sel, first, last):
    n = n_pos + nq - 1
    g, c, rng = _filled(ctx, fmt, H, hd, n, n + 1, 400 + n_pos % 100)
    q = rng.normal(size=(nq, H * G, hd)).astype(np.float32)
    idx = torch.full((nq, H, n_sel), 77, dtype=torch.int32, device="cuda")
    g.select(dev(q), idx, n_pos, n_first=first, n_last=last)
    want = ref.select(c, q, n_pos, n_sel, first, last)
    assert np.array_equal(host(idx), want)
    out = torch.empty((nq, H * G, hd), device="cuda")
    g.attend_blocks(dev(q), out, n_pos, idx)
    _check(host(out), *ref.attend_cache(c, q, n_pos, want))


@pytest.mark.parametrize("nq", [1, 3])
@pytest.mark.parametrize("n_blocks", [130, 2047, 15626, 60000])
def test_select_many_blocks(ctx, n_blocks, nq):
    """Random bounds and scales for up to 60,000 blocks (their keys no longer fit in shared memory), many equal
    scores, lists from one block to nearly all."""
    H, G, hd, n = 1, 3, 64, 64 * n_blocks - 5
    g, c = _cache(ctx, I8, H, hd, n + nq)
    rng = np.random.default_rng(n_blocks)
    a, b = rng.integers(-127, 128, size=(2, H, n_blocks, hd))
    c.kmin[:], c.kmax[:] = np.minimum(a, b), np.maximum(a, b)
    c.kmin[:, 40:90], c.kmax[:, 40:90] = c.kmin[:, 40:41], c.kmax[:, 40:41]
    c.scale["k"][:] = 2.0 ** rng.integers(-6, 3, size=(H, n_blocks))
    c.scale["k"][:, 40:90] = 4.0
    for name, v in (("kmin", c.kmin), ("kmax", c.kmax), ("kscale", c.scale["k"].astype(np.float32))):
        g.buffers[name].copy_(torch.from_numpy(v))
    q = rng.normal(size=(nq, H * G, hd)).astype(np.float32)
    for n_sel, first, last in ((1, 0, 0), (1, 1, 0), (17, 1, 4), (60, 0, 0), (n_blocks - 1, 2, 1), (128, 64, 64)):
        idx = torch.full((nq, H, n_sel), -9, dtype=torch.int32, device="cuda")
        g.select(dev(q), idx, n, n_first=first, n_last=last)
        assert np.array_equal(host(idx), ref.select(c, q, n, n_sel, first, last)), (n_sel, first, last)


def test_select_ties_and_odd_queries(ctx):
    """Equal blocks: ties go to the lowest index; q of zeros, NaN and infinities still gives a full, valid list."""
    H, G, hd, n = 1, 2, 64, 64 * 40
    g, c = _cache(ctx, I8, H, hd, n)
    x = np.tile(_rows(np.random.default_rng(16), 64, H, hd), (40, 1, 1))
    x[64 * 9:64 * 10] *= 2
    g.append(dev(x), dev(x), 0)
    c.append(x, x, 0)
    idx = torch.empty((1, H, 6), dtype=torch.int32, device="cuda")
    for kind in ("plain", "zero", "nan", "inf"):
        q = np.random.default_rng(17).normal(size=(1, G, hd)).astype(np.float32)
        if kind == "zero":
            q[:] = 0
        if kind == "nan":
            q[0, 0, :5] = np.nan
        if kind == "inf":
            q[0, 1, 3], q[0, 1, 4] = np.inf, -np.inf
        g.select(dev(q), idx, n, n_first=0, n_last=1)
        assert np.array_equal(host(idx), ref.select(c, q, n, 6, 0, 1)), kind


@pytest.mark.parametrize("fmt", [I8, E4M3])
def test_block_lists(ctx, fmt):
    """Lists of any order: skipped entries (negative, past the end), a block twice, an empty list (zeros), every block."""
    H, G, hd, n = 2, 4, 128, 64 * 6 + 9
    g, c, rng = _filled(ctx, fmt, H, hd, n + 1, n + 40, 18)
    q = rng.normal(size=(2, H * G, hd)).astype(np.float32)
    lists = np.array([[[5, 0, 6, -1, 2, 7, 100000, -2 ** 31], [-1] * 8],
                      [[3, 3, 3, 1, 2 ** 31 - 1, -5, 7, 3], [0, 1, 2, 3, 4, 5, 6, 7]]], dtype=np.int32)
    out = torch.full((2, H * G, hd), 4.0, device="cuda")
    g.attend_blocks(dev(q), out, n, dev(lists))
    want, tol = ref.attend_cache(c, q, n, lists)
    _check(host(out), want, tol)
    assert not host(out)[0, G:].any()
    whole = torch.empty_like(out)
    g.attend(dev(q), whole, n)
    _check(host(out)[1, G:], host(whole)[1, G:].astype(np.float64), 2 * tol[1, G:])


# ---- as they are used together ----------------------------------------------------------------
@pytest.mark.parametrize("fmt", [I8, E4M3])
def test_decode_run(ctx, fmt):
    """A prompt, then decode steps: append, attend, select, attend to the chosen blocks, all enqueued on one stream
    without a sync in between; each step against the oracle."""
    H, G, hd, prompt, steps, n_sel = 2, 4, 128, 250, 140, 4
    rng = np.random.default_rng(19)
    stride = prompt + steps
    g, c = _cache(ctx, fmt, H, hd, stride)
    k, v = _rows(rng, stride, H, hd, 1.0), _rows(rng, stride, H, hd, 1.0)
    q = rng.normal(size=(steps, 1, H * G, hd)).astype(np.float32)
    kd, vd, qd = dev(k), dev(v), dev(q)
    outs = torch.empty((2, steps, 1, H * G, hd), device="cuda")
    idx = torch.empty((steps, 1, H, n_sel), dtype=torch.int32, device="cuda")
    g.append(kd[:prompt], vd[:prompt], 0)
    for t in range(steps):
        p = prompt + t
        g.append(kd[p:p + 1], vd[p:p + 1], p)
        g.attend(qd[t], outs[0, t], p + 1)
        g.select(qd[t], idx[t], p + 1, n_first=1, n_last=1)
        g.attend_blocks(qd[t], outs[1, t], p + 1, idx[t])
    ctx.sync()
    o, ix = host(outs), host(idx)
    c.append(k[:prompt], v[:prompt], 0)
    for t in range(steps):
        p = prompt + t
        c.append(k[p:p + 1], v[p:p + 1], p)
        if t % 13 and p % 64 not in (0, 63):
            continue
        _check(o[0, t], *ref.attend_cache(c, q[t], p + 1))
        want = ref.select(c, q[t], p + 1, n_sel, 1, 1)
        assert np.array_equal(ix[t], want)
        _check(o[1, t], *ref.attend_cache(c, q[t], p + 1, want))
    _same(g, c, stride)


@pytest.mark.parametrize("capacity", [200, 3000, 20000])
def test_captured_step_replays_with_a_device_position(ctx, capacity):
    """One CUDA graph of a whole step (append, attend, select, attend to blocks) replayed while the position moves on
    the device (the launches are sized by the capacity: one CTA a head, a cluster, two launches); past the cache's
    end it writes nothing and the sync reports it."""
    _, nt = _mods()
    H, G, hd, n_sel, steps = 2, 4, 128, 3, 80
    stride, start = capacity, capacity - steps
    if capacity > 200:  # short at first, then at the end
        start = 120
    g, c, rng = _filled(ctx, I8, H, hd, start, stride, 20)
    k, v = _rows(rng, steps, H, hd), _rows(rng, steps, H, hd)
    q = rng.normal(size=(steps, 1, H * G, hd)).astype(np.float32)
    pos = torch.tensor([start], dtype=torch.int64, device="cuda")
    kb, vb = torch.empty((1, H, hd), device="cuda"), torch.empty((1, H, hd), device="cuda")
    qb, ob, sb = (torch.empty((1, H * G, hd), device="cuda") for _ in range(3))
    ib = torch.empty((1, H, n_sel), dtype=torch.int32, device="cuda")

    def step():
        g.append(kb, vb, 0, pos_dev=pos)
        g.attend(qb, ob, 0, pos_dev=pos)
        g.select(qb, ib, 0, n_first=0, n_last=1, pos_dev=pos)
        g.attend_blocks(qb, sb, 0, ib, pos_dev=pos)

    def compare(t, n):
        _check(host(ob), *ref.attend_cache(c, q[t], n))
        want = ref.select(c, q[t], n, n_sel, 0, 1)
        assert np.array_equal(host(ib), want)
        _check(host(sb), *ref.attend_cache(c, q[t], n, want))

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in range(steps):
        kb.copy_(dev(k[t:t + 1])), vb.copy_(dev(v[t:t + 1])), qb.copy_(dev(q[t]))
        graph.replay()
        c.append(k[t:t + 1], v[t:t + 1], start + t)
        if t % 9 == 0 or t == steps - 1:
            compare(t, start + t + 1)
        pos += 1
    if capacity > 200:  # the rest of the cache at once, with rows at a device position; the last position by replay
        m = stride - start - steps - 1
        km, vm = _rows(rng, m, H, hd), _rows(rng, m, H, hd)
        g.append(dev(km), dev(vm), 0, pos_dev=pos)
        c.append(km, vm, start + steps)
        pos += m
        graph.replay()
        c.append(k[steps - 1:], v[steps - 1:], stride - 1)
        compare(steps - 1, stride)
    ctx.sync()
    before = {n: b.clone() for n, b in g.buffers.items()}
    for bad in (stride, -1, 2 ** 62):
        pos.fill_(bad)
        graph.replay()
        with pytest.raises(nt.NtError):
            ctx.sync()
    for n, b in g.buffers.items():
        assert torch.equal(b.view(torch.uint8), before[n].view(torch.uint8)), n
    ctx.sync()


@pytest.mark.parametrize("n,nq", [(200, 1), (1000, 1), (20000, 1), (3000, 3), (3000, 7)])
def test_stalled_copies_are_reported(ctx, n, nq):
    """Bounded waits: with the copies held back (the test hook) the attention gives up, the sync reports a timeout, and
    the next call on the context is right (one CTA a head, a cluster, two launches, more rows than a warp's 8)."""
    _, nt = _mods()
    H, G, hd = 2, 4, 128
    g, c, rng = _filled(ctx, I8, H, hd, n + nq - 1, n + nq - 1, 25)
    q = rng.normal(size=(nq, H * G, hd)).astype(np.float32)
    out = torch.empty((nq, H * G, hd), device="cuda")
    idx = torch.arange(ref.blocks(n + nq), dtype=torch.int32, device="cuda").repeat(nq, H, 1).contiguous()
    for call in (lambda: g.attend(dev(q), out, n), lambda: g.attend_blocks(dev(q), out, n, idx)):
        nt.nt_debug_stall_waits(1)
        try:
            call()
        finally:
            nt.nt_debug_stall_waits(0)
        with pytest.raises(nt.NtError) as e:
            ctx.sync()
        assert e.value.status == nt.NT_ERR_TIMEOUT
        call()
        ctx.sync()
        _check(host(out), *ref.attend_cache(c, q, n))


def test_rewriting_rows_changes_nothing(ctx):
    """The same rows written again at the same positions: the scales and bytes stay."""
    rng = np.random.default_rng(26)
    g, c = _cache(ctx, E4M3, 2, 64, 300)
    k, v = _rows(rng, 200, 2, 64, 2.0), _rows(rng, 200, 2, 64)
    g.append(dev(k), dev(v), 0)
    g.append(dev(k[70:]), dev(v[70:]), 70)
    c.append(k, v, 0)
    c.append(k[70:], v[70:], 70)
    before = {n: host(b).copy() for n, b in g.buffers.items()}
    _same(g, c, 200)
    g.append(dev(k[70:]), dev(v[70:]), 70)
    for n, b in g.buffers.items():
        assert np.array_equal(host(b), before[n], equal_nan=b.dtype == torch.float32), n


def test_output_in_place_of_q(ctx):
    """out may be q itself, whatever the number of splits."""
    for n, nq in ((100, 1), (1000, 3), (9000, 1), (9000, 8)):
        g, c, rng = _filled(ctx, I8, 2, 128, n + nq - 1, n + nq, 27)
        q = rng.normal(size=(nq, 8, 128)).astype(np.float32)
        x = dev(q)
        g.attend(x, x, n)
        _check(host(x), *ref.attend_cache(c, q, n))


def test_streams_and_contexts(ctx):
    """Two contexts on two streams at once, each ordered on its own stream behind the work that makes its inputs."""
    _, nt = _mods()
    H, G, hd, n = 2, 4, 128, 3001
    other = nt.Context(0)
    try:
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        sets = []
        for cx, st, seed in ((ctx, streams[0], 21), (other, streams[1], 22)):
            g, c, rng = _filled(cx, E4M3, H, hd, n, n, seed)
            q = rng.normal(size=(1, H * G, hd)).astype(np.float32)
            sets.append((g, c, q, st, dev(q), torch.zeros((20, 1, H * G, hd), device="cuda")))
        torch.cuda.synchronize()
        for i in range(20):
            for g, c, q, st, qd, out in sets:
                with torch.cuda.stream(st):
                    scaled = qd * 1.0
                    g.attend(scaled, out[i], n)
        torch.cuda.synchronize()
        for g, c, q, st, qd, out in sets:
            want, tol = ref.attend_cache(c, q, n)
            for i in range(20):
                _check(host(out[i]), want, tol)
    finally:
        other.close()


def test_offsets_past_32_bits(ctx):
    """Two heads of 2^25 + 200 positions: the second head's rows lie past 2^32 bytes."""
    engine, _ = _mods()
    H, G, hd, fmt = 2, 2, 128, I8
    stride = 2 ** 25 + 200
    g = engine.KV8Cache(ctx, fmt, H, hd, stride, bounds=False)
    c = ref.Cache(fmt, H, hd, 300)
    rng = np.random.default_rng(23)
    base = (stride - 300) // 64 * 64
    k, v = _rows(rng, 300, H, hd), _rows(rng, 300, H, hd)
    g.append(dev(k), dev(v), base)
    c.append(k, v, 0)
    back = torch.empty(H, 300, hd, device="cuda")
    g.read(base, back, torch.empty_like(back))
    assert np.array_equal(host(back), c.read("k", np.arange(300)).astype(np.float32))
    q = rng.normal(size=(1, H * G, hd)).astype(np.float32)
    first = base // 64
    nb = ref.blocks(base + 300) - first
    idx = torch.arange(first, first + nb, dtype=torch.int32, device="cuda").repeat(1, H, 1).contiguous()
    out = torch.empty((1, H * G, hd), device="cuda")
    g.attend_blocks(dev(q), out, base + 300, idx)
    _check(host(out), *ref.attend_cache(c, q, 300))


def test_guards(ctx):
    """Outputs next to canaries: nothing outside them is written."""
    H, G, hd, n, nq, n_sel = 3, 5, 64, 333, 3, 4
    g, c, rng = _filled(ctx, E4M3, H, hd, n + nq - 1, n + nq - 1, 24)
    q = dev(rng.normal(size=(nq, H * G, hd)).astype(np.float32))
    buf = torch.full((nq * H * G * hd + 64,), 3.0, device="cuda")
    out = buf[32:-32].view(nq, H * G, hd)
    ib = torch.full((nq * H * n_sel + 64,), 11, dtype=torch.int32, device="cuda")
    idx = ib[32:-32].view(nq, H, n_sel)
    rb = torch.full((H * n * hd + 64,), 3.0, device="cuda")
    back = rb[32:-32].view(H, n, hd)
    g.attend(q, out, n)
    g.select(q, idx, n)
    g.attend_blocks(q, out, n, idx)
    g.read(0, back, back)
    torch.cuda.synchronize()
    for b, val in ((buf, 3.0), (ib, 11), (rb, 3.0)):
        assert bool((b[:32] == val).all()) and bool((b[-32:] == val).all())
