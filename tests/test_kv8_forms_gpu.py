"""Attention over the 8-bit cache in every launch form (rows per warp, step
length, one CTA a head, a cluster, two launches), at sizes where each warp takes
several steps, and block selection in every form of its choice."""
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


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _cache(ctx, fmt, H, hd, n, seed):
    """A cache of random bytes and scales, as if quantised before: device and oracle; the last rows' block is ragged."""
    from block_quantized_gemv_nt_gb300 import engine
    rng = np.random.default_rng(seed)
    g, c = engine.KV8Cache(ctx, fmt, H, hd, n), ref.Cache(fmt, H, hd, n)
    for w in "kv":
        if fmt == I8:
            b = np.clip(np.rint(rng.normal(size=(H, n, hd)) * 32), -127, 127).astype(np.int8).view(np.uint8)
        else:
            b = rng.integers(0, 256, size=(H, n, hd), dtype=np.uint8)
            b[(b & 0x7F) > 0x72] ^= 0x40  # up to 160; no NaN
        unit = 2.0 ** -5 if fmt == I8 else 2.0 ** -6
        c.data[w] = b
        c.scale[w] = unit * 2.0 ** rng.integers(-1, 2, size=c.scale[w].shape)
        g.buffers[w].copy_(torch.from_numpy(b))
        g.buffers[w + "scale"].copy_(torch.from_numpy(c.scale[w].astype(np.float32)))
    return g, c, rng


DENSE = [  # form, H, G, hd, n_pos, nq, format
    (dict(R=1, U=2, cluster=False), 8, 4, 128, 16384, 1, I8),
    (dict(R=1, U=2, cluster=False), 8, 4, 128, 32769, 1, E4M3),
    (dict(R=1, U=2, cluster=False), 2, 7, 64, 131071, 1, E4M3),
    (dict(R=1, U=2, cluster=False), 2, 4, 128, 131071, 1, I8),
    (dict(R=1, U=2, cluster=False), 8, 1, 64, 40000, 5, I8),
    (dict(R=1, U=1, cluster=False), 2, 4, 128, 20001, 1, E4M3),
    (dict(R=1, U=2, cluster=True), 2, 4, 128, 12000, 1, I8),
    (dict(R=1, U=2, cluster=True), 8, 4, 128, 10300, 1, E4M3),
    (dict(R=1, U=2, cluster=True), 3, 5, 64, 6100, 1, I8),
    (dict(R=1, U=1, cluster=True), 8, 8, 128, 9001, 1, I8),
    (dict(R=2, U=2, cluster=True), 2, 4, 128, 12281, 8, I8),
    (dict(R=2, U=2, cluster=False), 8, 4, 128, 16381, 8, E4M3),
    (dict(R=2, U=2, cluster=False), 2, 4, 128, 16381, 8, I8),
    (dict(R=2, U=2, cluster=False), 2, 3, 64, 40003, 7, E4M3),
    (dict(R=2, U=2, cluster=False), 1, 16, 128, 30000, 1, I8),
    (dict(R=2, U=2, cluster=False), 4, 16, 64, 5000, 16, I8),
]


def _is_form(p, form):
    assert all(p[x] == form[x] for x in form), (p, form)
    assert p["S"] > 1


@pytest.mark.parametrize("form,H,G,hd,n_pos,nq,fmt", DENSE)
def test_attention_forms(ctx, form, H, G, hd, n_pos, nq, fmt):
    if _sms() != 152:
        pytest.skip("the sizes reach these forms on 152 SMs")
    p = tight.plan(_sms(), H, G, hd, nq, n_pos)
    _is_form(p, form)
    g, c, rng = _cache(ctx, fmt, H, hd, n_pos + nq - 1, n_pos + hd)
    q = rng.normal(size=(nq, H * G, hd)).astype(np.float32)
    out = torch.empty((nq, H * G, hd), device="cuda")
    g.attend(dev(q), out, n_pos)
    ctx.sync()
    tight.check(host(out), c, q, n_pos, p)
    again = torch.empty_like(out)
    g.attend(dev(q), again, n_pos)
    assert torch.equal(out, again)


def test_attention_of_a_million_positions(ctx):
    """1,000,003 positions of one head: 13 steps a warp, 304 splits."""
    H, G, hd, n = 1, 4, 64, 1000003
    g, c, rng = _cache(ctx, I8, H, hd, n, 5)
    q = rng.normal(size=(1, H * G, hd)).astype(np.float32)
    out = torch.empty((1, H * G, hd), device="cuda")
    g.attend(dev(q), out, n)
    ctx.sync()
    tight.check(host(out), c, q, n, tight.plan(_sms(), H, G, hd, 1, n))


SPARSE = [  # form, H, G, hd, n_pos, nq, n_sel, format
    (dict(R=1, U=2, cluster=False), 8, 4, 128, 16384 + 33, 5, 64, E4M3),
    (dict(R=1, U=2, cluster=False), 8, 4, 128, 60001, 1, 500, I8),
    (dict(R=1, U=2, cluster=True), 8, 4, 64, 30001, 3, 88, I8),
    (dict(R=1, U=1, cluster=True), 8, 4, 128, 20001, 1, 128, I8),
    (dict(R=2, U=2, cluster=True), 2, 12, 128, 5003, 1, 30, E4M3),
    (dict(R=2, U=2, cluster=True), 1, 16, 64, 5003, 3, 9, I8),
    (dict(R=2, U=2, cluster=False), 2, 9, 128, 60001, 1, 300, I8),
    (dict(R=2, U=2, cluster=False), 4, 11, 64, 30001, 4, 60, E4M3),
]


@pytest.mark.parametrize("form,H,G,hd,n_pos,nq,n_sel,fmt", SPARSE)
def test_block_attention_forms(ctx, form, H, G, hd, n_pos, nq, n_sel, fmt):
    if _sms() != 152:
        pytest.skip("the sizes reach these forms on 152 SMs")
    p = tight.plan(_sms(), H, G, hd, nq, n_pos, n_sel)
    _is_form(p, form)
    g, c, rng = _cache(ctx, fmt, H, hd, n_pos + nq - 1, n_pos + hd)
    q = rng.normal(size=(nq, H * G, hd)).astype(np.float32)
    nb = ref.blocks(n_pos)
    lists = np.stack([[np.sort(rng.choice(nb, n_sel, replace=False)) for _ in range(H)] for _ in range(nq)])
    lists[..., -1] = nb - 1       # the ragged last block,
    lists[..., n_sel // 3] = -1   # an entry to skip,
    lists[0, 0] = lists[0, 0][rng.permutation(n_sel)]  # any order
    out = torch.empty((nq, H * G, hd), device="cuda")
    g.attend_blocks(dev(q), out, n_pos, dev(lists.astype(np.int32)))
    ctx.sync()
    tight.check(host(out), c, q, n_pos, p, lists)


@pytest.mark.parametrize("hd,H,nq,n_blocks", [(64, 2, 1, 257), (128, 2, 2, 1024), (64, 1, 1, 5120), (64, 1, 1, 17408),
                                              (64, 2, 1, 17409), (64, 1, 2, 30000), (128, 1, 1, 54784), (64, 1, 1, 54785)])
def test_selection_forms(ctx, hd, H, nq, n_blocks):
    """Every form of the choice and its borders (keys in registers by 1 and 5, re-read from shared memory, in
    scratch), each call many times: the list is exact every time and nothing beside it is written."""
    G, n = 3, 64 * n_blocks - 63
    rng = np.random.default_rng(n_blocks)
    from block_quantized_gemv_nt_gb300 import engine
    g, c = engine.KV8Cache(ctx, I8, H, hd, n + nq), ref.Cache(I8, H, hd, n + nq)
    nb = c.kmin.shape[1]
    a, b = rng.integers(-127, 128, size=(2, H, nb, hd))
    c.kmin[:], c.kmax[:] = np.minimum(a, b), np.maximum(a, b)
    c.scale["k"][:] = 2.0 ** rng.integers(-6, 3, size=(H, nb))
    for name, v in (("kmin", c.kmin), ("kmax", c.kmax), ("kscale", c.scale["k"].astype(np.float32))):
        g.buffers[name].copy_(torch.from_numpy(v))
    q = rng.normal(size=(nq, H * G, hd)).astype(np.float32)
    qd = dev(q)
    for n_sel, first, last in ((1, 0, 0), (65, 1, 4), (n_blocks // 2, 0, 1)):
        want = ref.select(c, q, n, n_sel, first, last)
        size = nq * H * n_sel
        buf = torch.full((40, size + 64), -9, dtype=torch.int32, device="cuda")
        for i in range(40):
            g.select(qd, buf[i, 32:32 + size].view(nq, H, n_sel), n, n_first=first, n_last=last)
        got = host(buf)
        assert np.all(got[:, :32] == -9) and np.all(got[:, 32 + size:] == -9)
        assert np.all(got[:, 32:32 + size] == want.reshape(1, -1)), (n_sel, first, last)
