"""Attention over the paged 4-bit cache where one position takes nearly all of the weight and
its V is 0: the output is what many weights 2^-16 to 2^-30 of the largest give together."""
import math

import numpy as np
import pytest

import kv4_ref as ref
from gpu_util import dev, host, need_gpu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from block_quantized_gemv_nt_gb300 import engine, nt  # noqa: E402


@pytest.fixture(scope="module")
def ctx():
    need_gpu()
    c = nt.Context(0)
    yield c
    c.close()


def expect(q, k, v):
    """q [rows][Hq][hd], all of k, v [n][H][hd], the rows the last of them -> (out, bound on its error).

    With A_j = sum_d |q_d k_jd| / sqrt(hd), a position's score is off by A_j 2^-18.5 (the products' roundings, as in
    kv4_ref.attend), its weight by that much; the sum of the weights by the weights' mean of it.  Every weight shares 2^-19
    (ex2, the tensor cores' steps, divisions), the largest A times 2^-21 (the maximum and the distance from it, rounded),
    and 2^-23 for each 64 positions.  A weight's two parts leave out 2^-22 of it, within the 2^-19, or, where the lower one
    ends at f16's least step, half of that over 2^11, 2^-36, where the largest weight stands at 2^8 or above: 2^-44 of it."""
    n_q, Hq, hd = q.shape
    n, H = k.shape[:2]
    out, bound = np.zeros((n_q, Hq, hd)), np.zeros((n_q, Hq, hd))
    for i in range(n_q):
        m = n - (n_q - 1 - i)
        for h in range(Hq):
            kk, vv, x = k[:m, h * H // Hq], v[:m, h * H // Hq], q[i, h]
            s = kk @ x / math.sqrt(hd)
            w = np.exp(s - s.max())
            w /= w.sum()
            A = np.abs(kk) @ np.abs(x) / math.sqrt(hd)
            d = A * 2.0 ** -18.5 + 2.0 ** -19 + A.max() * 2.0 ** -21 + (m / 64 + 1) * 2.0 ** -23
            out[i, h] = w @ vv
            bound[i, h] = (w * d) @ np.abs(vv) + np.abs(out[i, h]) * (w @ d) + 2.0 ** -44 * w.max() * np.abs(vv).sum(axis=0)
    return out, bound


@pytest.mark.parametrize("fmt", [nt.KV4_I4, nt.KV4_E2M1])
@pytest.mark.parametrize("tail", ["equal", "spread"])
@pytest.mark.parametrize("binades", [16, 20, 23, 26, 30])
@pytest.mark.parametrize("hd,H,G,n,rows", [(128, 2, 4, 64, 1), (64, 2, 8, 64, 3), (128, 1, 1, 900, 1), (64, 1, 2, 1500, 1500)])
def test_one_position_takes_the_weight_and_gives_nothing(ctx, fmt, tail, binades, hd, H, G, n, rows):
    rng = np.random.default_rng(binades)
    k, v = np.zeros((n, H, hd)), rng.uniform(0.5, 1.5, (n, H, hd))
    if tail == "spread":
        k[:, :, 1:] = 0.5 * rng.standard_normal((n, H, hd - 1))
    k[0], v[0] = 0, 0
    k[0, :, 0] = binades * math.log(2) * math.sqrt(hd) / 8
    q = rng.standard_normal((rows, H * G, hd))
    q[:, :, 0] = 8
    q, k, v = q.astype(np.float32), k.astype(np.float32), v.astype(np.float32)
    pages = -(-n // 64)
    cache = engine.KV4Cache(ctx, fmt, H, hd, pages)
    cache.append(dev(k), dev(v), torch.arange(n, device="cuda"))
    out = torch.empty(rows, H * G, hd, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cache.attend(dev(q), out, i32(0, rows), i32(n), torch.arange(pages, dtype=torch.int32, device="cuda")[None])
    ctx.sync()
    want, bound = expect(q.astype(np.float64), ref.values(k, fmt), ref.values(v, fmt))
    off = np.abs(host(out) - want)
    assert (off <= bound).all(), float((off / np.maximum(bound, 1e-300)).max())
