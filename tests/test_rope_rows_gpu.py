"""Rotary positions of rows (nt_rope_rows) against the 64-bit numpy oracle (kv4_ref)."""
import numpy as np
import pytest

import kv4_ref as ref
from gpu_util import dev, host, need_gpu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from block_quantized_gemv_nt_gb300 import engine, nt  # noqa: E402

KIND = {"plain": nt.ROPE_PLAIN, "linear": nt.ROPE_LINEAR, "base": nt.ROPE_BASE, "bands": nt.ROPE_BANDS,
        "ramp": nt.ROPE_RAMP}
ARGS = {"plain": {}, "linear": dict(factor=4.0), "base": dict(factor=8.0), "bands": dict(factor=8.0, old_len=8192.0),
        "ramp": dict(factor=16.0, old_len=4096.0)}


@pytest.fixture(scope="module")
def ctx():
    need_gpu()
    c = nt.Context(0)
    yield c
    c.close()


def _check(got, x, positions, freq, layout, mag, half):
    """|error| over the pair's length: the turn is off by 2^-33 of a turn and its fp32 rounding, 2^-24 of half a turn
    (2 pi 2^-25 = 1.9e-7), sincospi by an ulp or two (1.2e-7), the products and their sum by three roundings of 2^-24;
    the frequency's own double is off by a few 2^-53, times the position: 5e-7 in all up to positions of 2^30.  An F16
    output adds its rounding, 2^-11 of the value (2^-25 below f16's normal numbers)."""
    want = ref.rotate(x, positions, freq, layout, mag)
    r = 2 * len(freq)
    a, b = (slice(0, r, 2), slice(1, r, 2)) if layout == 0 else (slice(0, r // 2), slice(r // 2, r))
    size = np.zeros_like(want)
    size[..., a] = size[..., b] = mag * np.hypot(x[..., a], x[..., b])
    far = np.abs(np.asarray(positions, dtype=np.float64)).max(initial=0) * 16 * 2.0 ** -53
    bound = size * (5e-7 + far) + (np.abs(want) * 2.0 ** -11 + 2.0 ** -25 if half else 0)
    assert (np.abs(host(got).astype(np.float64) - want) <= bound).all()
    assert np.array_equal(host(got)[..., r:], x[..., r:].astype(host(got).dtype))


@pytest.mark.parametrize("layout", [nt.ROPE_PAIRS, nt.ROPE_HALVES])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("hd,rot", [(64, 64), (128, 128), (128, 96), (64, 8), (256, 256), (8, 8), (200, 56)])
@pytest.mark.parametrize("n,heads", [(1, (1,)), (5, (7, 2)), (33, (3, 1, 5))])
def test_rows(ctx, layout, dtype, hd, rot, n, heads):
    rng = np.random.default_rng(hd + rot + n)
    name = list(ARGS)[(hd // 8 + n) % 5]
    rope = engine.Rope(ctx, hd, rot, layout, theta=500000.0, scaling=KIND[name], **ARGS[name])
    freq = ref.frequencies(rot, 500000.0, name, **ARGS[name])
    pos = rng.integers(0, 200000, n).astype(np.int32)
    xs = [torch.from_numpy(rng.standard_normal((n, h, hd)).astype(np.float32)).to(dtype).cuda() for h in heads]
    keep = [host(x).astype(np.float64) for x in xs]
    ys = [torch.full_like(x, 99.0) for x in xs]
    rope.rotate(*zip(xs, ys), positions=dev(pos))
    for x, y, x0 in zip(xs, ys, keep):
        assert np.array_equal(host(x), x0.astype(host(x).dtype))
        _check(y, x0, pos, freq, layout, rope.plan.mag, dtype is torch.float16)
    rope.rotate(*[(x, x) for x in xs], positions=dev(pos))       # in place, the same bits
    for x, y in zip(xs, ys):
        assert np.array_equal(host(x), host(y))
    ctx.sync()


def test_far_positions(ctx):
    """Positions to the ends of 32 bits lose nothing: the angle is exact modulo a turn."""
    pos = np.array([0, 1, 2 ** 24 + 1, 2 ** 30 + 3, 2 ** 31 - 1, -1, -2 ** 31, 123456789], dtype=np.int32)
    x = np.random.default_rng(1).standard_normal((len(pos), 2, 64)).astype(np.float32)
    rope = engine.Rope(ctx, 64)
    y = torch.empty(len(pos), 2, 64, device="cuda")
    rope.rotate((dev(x), y), positions=dev(pos))
    # against the plan's own turns, in exact integers: what the frequencies' doubles round to is no part of this
    turns = np.array([[((int(p) * rope.plan.turns[i]) % 2 ** 64) / 2.0 ** 64 for i in range(32)] for p in pos])
    c, s = np.cos(2 * np.pi * turns)[:, None], np.sin(2 * np.pi * turns)[:, None]
    a, b = x[..., 0::2].astype(np.float64), x[..., 1::2].astype(np.float64)
    want = np.empty(x.shape)
    want[..., 0::2], want[..., 1::2] = a * c - b * s, a * s + b * c
    size = np.repeat(np.hypot(a, b), 2, axis=-1)
    assert (np.abs(host(y) - want) <= 5e-7 * size).all()


def test_there_and_back(ctx):
    """The turn of -p undoes that of p; magnitudes multiply."""
    rng = np.random.default_rng(2)
    x = rng.standard_normal((50, 3, 128)).astype(np.float32)
    pos = rng.integers(0, 1 << 20, 50).astype(np.int32)
    rope = engine.Rope(ctx, 128, 128, nt.ROPE_HALVES, mag=2.0)
    y = dev(x)
    rope.rotate((y, y), positions=dev(pos))
    rope.rotate((y, y), positions=dev(-pos))
    assert np.abs(host(y) / 4.0 - x).max() <= 1e-6 * np.hypot(x[..., :64], x[..., 64:]).max()


def test_as_the_one_position_call(ctx):
    """nt_rope's rows, one position at a time: same pairs, same frequencies."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 2, 64)).astype(np.float32)
    rope = engine.Rope(ctx, 64, theta=10000.0)
    y = dev(x)
    rope.rotate((y, y), pos0=1000)
    for i in range(4):
        z = dev(x[i])
        nt.nt_rope(ctx, z, None, 2, 0, 64, 1000 + i, 10000.0)
        assert np.abs(host(z) - host(y)[i]).max() <= 1e-6 * np.abs(x).max() * 2
    ctx.sync()


def test_strides_and_rows_between(ctx):
    """q and k inside one fused buffer, in place: the rows of v between and behind them stay."""
    rng = np.random.default_rng(4)
    buf = rng.standard_normal((9, 8, 64)).astype(np.float32)
    t = dev(buf)
    rope = engine.Rope(ctx, 64, 32, nt.ROPE_PAIRS)
    rope.rotate((t[:, :4], t[:, :4]), (t[:, 5:7], t[:, 5:7]), pos0=5)
    got, freq = host(t), ref.frequencies(32, 10000.0, "plain")
    _check(t[:, :4], buf[:, :4].astype(np.float64), np.arange(5, 14), freq, 0, 1.0, False)
    _check(t[:, 5:7], buf[:, 5:7].astype(np.float64), np.arange(5, 14), freq, 0, 1.0, False)
    assert np.array_equal(got[:, 4], buf[:, 4]) and np.array_equal(got[:, 7], buf[:, 7])
    by_head = dev(buf).transpose(0, 1)             # [heads][n] seen as rows of 9 heads
    y = torch.empty(8, 9, 64, device="cuda")
    rope.rotate((by_head, y), pos0=3)
    _check(y, buf.transpose(1, 0, 2).astype(np.float64), np.arange(3, 11), freq, 0, 1.0, False)


def test_one_row_for_all(ctx):
    """An input broadcast over rows and heads (strides of 0), turned at each row's position; no rows at all."""
    x = np.random.default_rng(5).standard_normal((1, 1, 64)).astype(np.float32)
    y = torch.empty(7, 3, 64, device="cuda")
    rope = engine.Rope(ctx, 64, layout=nt.ROPE_HALVES)
    pos = np.array([0, 5, 5, 1, 70000, -3, 2], dtype=np.int32)
    rope.rotate((dev(x).expand(7, 3, 64), y), positions=dev(pos))
    _check(y, np.broadcast_to(x, (7, 3, 64)).astype(np.float64), pos, ref.frequencies(64, 10000.0, "plain"), 1, 1.0, False)
    with pytest.raises(nt.NtError):               # an output that is broadcast has no place for its rows
        rope.rotate((y, dev(x).expand(7, 3, 64)), positions=dev(pos))
    rope.rotate((y[:0], y[:0]), pos0=3)
    ctx.sync()


def test_not_finite_values_stay_in_their_pair(ctx):
    x = np.ones((1, 1, 64), dtype=np.float32)
    x[0, 0, 10], x[0, 0, 20] = np.nan, np.inf
    y = torch.empty(1, 1, 64, device="cuda")
    engine.Rope(ctx, 64).rotate((dev(x), y), pos0=3)
    bad = ~np.isfinite(host(y)[0, 0])
    assert set(np.flatnonzero(bad)) <= {10, 11, 20, 21} and bad[10] and bad[20]


def test_refusals(ctx):
    rope = engine.Rope(ctx, 64)
    x, pos = torch.zeros(4, 2, 64, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    for rows, kw in [([(x, x.half())], {}), ([(x, x[:2])], {}), ([(x.double(), x.double())], {}), ([(x[..., :32], x[..., :32])], {}),
                     ([(x, x)] * 4, {}), ([(x, x)], dict(positions=pos.long())), ([(x, x)], dict(positions=pos[:3])),
                     ([(x.cpu(), x.cpu())], {}), ([(x, x), (x[:3], x[:3])], {})]:
        with pytest.raises(ValueError):
            rope.rotate(*rows, **kw)

    def call(plan=rope.plan, fmt=nt.F32, n_jobs=1, n=4, pos0=0, positions=None, **job):
        j = (nt.nt_rope_job * 1)(nt.nt_rope_job(**{**dict(x_dev=x.data_ptr(), y_dev=x.data_ptr(), n_heads=2, x_tok_stride=128,
                                                         x_head_stride=64, y_tok_stride=128, y_head_stride=64), **job}))
        nt.nt_rope_rows(ctx, plan, fmt, j, n_jobs, n, positions, pos0)

    wrong = nt.nt_rope_plan()
    for kw in [dict(plan=wrong), dict(plan=None), dict(fmt=nt.Q8_0), dict(n_jobs=0), dict(n_jobs=4), dict(n=-1),
               dict(n=(1 << 24) + 1), dict(pos0=1 << 31), dict(pos0=-(1 << 31) - 1), dict(positions=pos.data_ptr() + 2),
               dict(x_dev=None), dict(y_dev=None), dict(n_heads=0), dict(n_heads=1025), dict(x_tok_stride=126),
               dict(y_head_stride=32), dict(y_tok_stride=64), dict(x_tok_stride=256), dict(x_dev=x.data_ptr() + 4),
               dict(x_tok_stride=1 << 41)]:
        with pytest.raises(nt.NtError) as e:
            call(**kw)
        assert e.value.status in (nt.NT_ERR_INVALID_ARG, nt.NT_ERR_ALIGNMENT, nt.NT_ERR_UNSUPPORTED_FMT), kw
    call(n=0)
    rope.rotate((x[:0], x[:0]))
    ctx.sync()


def test_captured(ctx):
    rng = np.random.default_rng(5)
    x, pos = torch.zeros(6, 2, 64, device="cuda"), torch.zeros(6, dtype=torch.int32, device="cuda")
    y = torch.empty_like(x)
    rope = engine.Rope(ctx, 64, 64, nt.ROPE_HALVES)
    rope.rotate((x, y), positions=pos)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rope.rotate((x, y), positions=pos)
    for i in range(3):
        data, p = rng.standard_normal(x.shape).astype(np.float32), rng.integers(0, 9999, 6).astype(np.int32)
        x.copy_(torch.from_numpy(data)), pos.copy_(torch.from_numpy(p))
        graph.replay()
        _check(y, data.astype(np.float64), p, ref.frequencies(64, 10000.0, "plain"), 1, 1.0, False)
