"""Pins of the 64-bit oracle of the paged 4-bit cache (kv4_ref), the rope plan's host
arithmetic, and what the binding refuses (CPU only)."""
import math
from fractions import Fraction

import numpy as np
import pytest

import kv4_ref as ref
from block_quantized_gemv_nt_gb300 import engine, nt

torch = pytest.importorskip("torch")


def test_page_bytes():
    assert nt.nt_kv4_layout(128) == 2 * (64 * 64 + 64 * 4 * 2)
    assert nt.nt_kv4_layout(64) == 2 * (64 * 32 + 64 * 2 * 2)
    for hd in (0, 32, 96, 256):
        with pytest.raises(nt.NtError):
            nt.nt_kv4_layout(hd)


def test_i4_by_hand():
    x = np.zeros(32)
    x[:8] = [-8.0, 7.0, 7.5, 3.5, 2.5, -2.5, -0.5, 0.5]   # the scale is 1: -8 is the largest
    assert ref.values(x, ref.I4)[:8].tolist() == [-8, 7, 7, 4, 2, -2, 0, 0]
    x[0] = 8.0                                            # the scale is -1
    assert ref.values(x, ref.I4)[:8].tolist() == [8, 7, 8, 4, 2, -2, 0, 0]
    x[:2] = [-8.0, 8.0]                                   # two that tie: the positive one is exact
    assert ref.values(x, ref.I4)[:2].tolist() == [-7, 8]


def test_e2m1_by_hand():
    x = np.zeros(32)
    x[:16] = [6, 5, 5.001, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, 0.2501, -0.25, -0.75, -1.75, -2.5, -3.5, -5]
    want = [6, 4, 6, 4, 2, 2, 1, 1, 0, 0.5, 0, -1, -2, -2, -4, -4]
    assert ref.values(x, ref.E2M1)[:16].tolist() == want


def test_scales_have_8_bits():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((400, 1, 32)) * np.exp(rng.uniform(-12, 8, (400, 1, 1)))
    for fmt in (ref.I4, ref.E2M1):
        d = ref.scales(x, fmt)
        assert np.array_equal(d, d.astype(np.float16).astype(np.float64))
        m, _ = np.frexp(d)
        assert np.array_equal(m * 256, np.round(m * 256))
        top = np.abs(x).max(axis=-1) / (8 if fmt == ref.I4 else 6)
        ok = np.abs(np.abs(d) - np.minimum(top, ref.TOP_SCALE)) <= np.maximum(top * 2.0 ** -8, 2.0 ** -24)
        assert ok.all()


def test_largest_scale():
    x = np.full(32, 1e30)
    assert ref.values(x, ref.I4).max() == 8 * 2720 and ref.values(x, ref.E2M1).max() == 6 * 2720


def test_attention_by_hand():
    k = np.zeros((3, 1, 64))
    v = np.arange(3.0)[:, None, None] + np.zeros((3, 1, 64))
    out, _ = ref.attend(np.ones((2, 2, 64)), k, v, 2)     # the first of two rows sees two positions
    assert np.allclose(out[0], 0.5) and np.allclose(out[1], 1.0)
    out, _ = ref.attend(np.ones((4, 1, 64)), k, v, 4)     # the first of four rows of three positions sees none
    assert np.array_equal(out[0], np.zeros((1, 64)))


def test_pages_by_hand():
    table = [[5, 0], [7, 0], [0, 0]]
    held, free = [64, 10, 0], [1, 2, 3, 0, 0, 0, 0, 0]
    n, q, slots, pos, wrong = ref.pages_step(table, held, [64, 0, 0], [1, 0, 2], free, 3, 8, 4)
    # request 1 gives 7 back, request 0 takes it, request 2 takes 3
    assert (n, q, slots, pos, wrong) == (2, [0, 1, 1, 3], [7 * 64, 3 * 64, 3 * 64 + 1, -1], [64, 0, 1, 0], False)
    assert held == [65, 0, 2] and table == [[5, 7], [7, 0], [3, 0]]


# ---- rope plans ------------------------------------------------------------------
PLANS = [("plain", {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
         ("bands", dict(factor=8.0, old_len=8192.0)), ("bands", dict(factor=32.0, old_len=4096.0, low=2.0, high=8.0)),
         ("ramp", dict(factor=16.0, old_len=4096.0)), ("ramp", dict(factor=4.0, old_len=32768.0, low=2.0, high=40.0))]
KIND = {"plain": nt.ROPE_PLAIN, "linear": nt.ROPE_LINEAR, "base": nt.ROPE_BASE, "bands": nt.ROPE_BANDS,
        "ramp": nt.ROPE_RAMP}


@pytest.mark.parametrize("rot", [8, 56, 128, 256])
@pytest.mark.parametrize("name,args", PLANS)
def test_plan_turns(name, args, rot):
    plan = nt.nt_rope_plan_init(256, rot, nt.ROPE_HALVES, theta=500000.0, scaling=KIND[name], **args)
    freq = ref.frequencies(rot, 500000.0, name, **args)
    for i, w in enumerate(freq):
        turn = plan.turns[i] / 2.0 ** 64
        # both sides evaluate the formula in doubles: a few of their roundings apart
        assert abs(turn - w / (2 * math.pi)) <= 32 * 2.0 ** -53 * w / (2 * math.pi) + 2.0 ** -64
    assert all(plan.turns[i] == 0 for i in range(rot // 2, 128))
    mag = 0.1 * math.log(args["factor"]) + 1.0 if name == "ramp" else 1.0
    assert plan.mag == np.float32(mag)


def test_ramp_of_a_length_that_every_pair_turns_often_over():
    # all pairs turn more than 32 times over the old length: none is slowed down
    plan = nt.nt_rope_plan_init(64, 64, theta=100.0, scaling=nt.ROPE_RAMP, factor=4.0, old_len=1e9)
    plain = nt.nt_rope_plan_init(64, 64, theta=100.0)
    assert list(plan.turns) == list(plain.turns)
    # the pair that turns once lies behind the last one (64.4 of 64): the ramp is not cut short
    plan = nt.nt_rope_plan_init(128, 128, theta=10000.0, scaling=nt.ROPE_RAMP, factor=4.0, old_len=65536.0)
    a, b = 40, 65                                         # 64 ln(L / (2 pi 32)) / ln theta = 40.2, 64.3
    u = [10000.0 ** (-2.0 * i / 128) for i in range(64)]
    for i in range(64):
        k = min(1.0, max(0.0, (i - a) / (b - a)))
        assert Fraction(plan.turns[i], 2 ** 64) == pytest.approx(u[i] * (1 - 0.75 * k) / (2 * math.pi), rel=1e-13)


def test_plan_divisors_and_whole_turns():
    div = [2.0 ** (i - 3) for i in range(8)]
    plan = nt.nt_rope_plan_init(16, 16, theta=10000.0, divisors=div, mag=0.5)
    for i in range(8):
        w = 10000.0 ** (-2.0 * i / 16) / div[i]
        assert Fraction(plan.turns[i], 2 ** 64) == pytest.approx(w / (2 * math.pi) % 1.0, rel=1e-14)
    assert plan.mag == 0.5


@pytest.mark.parametrize("bad", [
    dict(head_dim=0), dict(head_dim=12), dict(head_dim=264), dict(rot_dim=0), dict(rot_dim=136), dict(rot_dim=12),
    dict(layout=2), dict(layout=-1), dict(scaling=5), dict(scaling=-1), dict(theta=0.0), dict(theta=-1.0),
    dict(theta=1.0), dict(theta=float("nan")), dict(theta=float("inf")), dict(mag=-1.0), dict(mag=float("nan")),
    dict(scaling=1, factor=0.0), dict(scaling=1, factor=float("nan")), dict(scaling=3, factor=2.0),
    dict(scaling=3, factor=2.0, old_len=4096.0, low=4.0, high=4.0), dict(scaling=4, factor=2.0, old_len=-1.0),
    dict(scaling=4, factor=2.0, old_len=4096.0, theta=0.5), dict(divisors=[1.0] * 63), dict(divisors=[0.0] * 64),
    dict(divisors=[float("nan")] * 64), dict(low=-1.0), dict(high=float("inf"))])
def test_plan_refusals(bad):
    args = dict(head_dim=128, rot_dim=128)
    args.update(bad)
    with pytest.raises(nt.NtError) as e:
        nt.nt_rope_plan_init(**args)
    assert e.value.status == nt.NT_ERR_INVALID_ARG


# ---- what the classes refuse before any call ----------------------------------------
def _cache(**kw):
    args = dict(ctx=None, fmt=nt.KV4_I4, n_kvh=2, head_dim=64, n_pages=3, device="cpu")
    args.update(kw)
    return engine.KV4Cache(**args)


def test_cache_refusals():
    good = torch.zeros(3, 2, 4608, dtype=torch.uint8)
    _cache(data=good)
    for bad in (good[:2], good.int(), good.transpose(0, 1).contiguous(), torch.zeros(3, 2, 9216, dtype=torch.uint8)[..., ::2]):
        with pytest.raises(ValueError):
            _cache(data=bad)
    with pytest.raises(nt.NtError):
        _cache(head_dim=96)


def test_row_refusals():
    c = _cache()
    k, s = torch.zeros(5, 2, 64), torch.zeros(5, dtype=torch.int64)
    bad = [(k, k[:4], s), (k.double(), k.double(), s), (k.half(), k, s), (k[:, :1], k[:, :1], s), (k, k, s.int()),
           (k, k, s[:4]), (k, k, torch.zeros(10, dtype=torch.int64)[::2]), (k[..., :32], k[..., :32], s),
           (k.to(torch.bfloat16), k.to(torch.bfloat16), s), (k, k.transpose(0, 1).contiguous().transpose(0, 1), s)]
    for args in bad:
        with pytest.raises(ValueError):
            c.append(*args)
        with pytest.raises(ValueError):
            c.read(*args)


def test_attend_refusals():
    c = _cache()
    q, qs, held, table = (torch.zeros(3, 4, 64), torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                          torch.zeros(2, 7, dtype=torch.int32))
    bad = [(q.half(), q, qs, held, table), (q, q[:2], qs, held, table), (q, q, qs[:2], held, table),
           (q, q, qs.long(), held, table), (q, q, qs, held[:1], table), (q, q, qs, held.long(), table),
           (q, q, qs, held, table.long()), (q, q, qs, held, table[:, ::2]), (q[..., :32], q[..., :32], qs, held, table),
           (q.transpose(0, 1), q, qs, held, table), (q, q.half(), qs, held, table)]
    for args in bad:
        with pytest.raises(ValueError):
            c.attend(*args)


def test_pages_refusals():
    p = engine.KV4Pages(None, 2, 7, 9, device="cpu")
    assert p.free.tolist() == list(range(8, -1, -1)) and p.n_free.tolist() == [9]
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    s = torch.zeros(4, dtype=torch.int64)
    bad = [(i32(3), i32(3), s, i32(4)), (i32(2), i32(2), s, i32(4)), (i32(2), i32(3), s.int(), i32(4)),
           (i32(2), i32(3), s, i32(3)), (i32(2).long(), i32(3), s, i32(4))]
    for args in bad:
        with pytest.raises(ValueError):
            p.step(*args)
    for kw in (dict(keep=i32(3)), dict(held_out=i32(1)), dict(n_free_out=i32(2)), dict(keep=i32(2).long())):
        with pytest.raises(ValueError):
            p.step(i32(2), i32(3), s, i32(4), **kw)
    with pytest.raises(ValueError):
        engine.KV4Pages(None, 2, 7, 9, buffers=dict(table=torch.zeros(2, 6, dtype=torch.int32), held=i32(2), free=i32(9),
                                                    n_free=i32(1)))
