"""The paged 4-bit KV cache, its tables, its attention and the rotary rows in plain
numpy, 64 bits: the oracle of test_kv4_gpu.py, test_kv4_pages_gpu.py and
test_rope_rows_gpu.py.  It shares no code with the library."""
import math

import numpy as np

PAGE, GROUP = 64, 32
I4, E2M1 = 0, 1
TOP_SCALE = 2720.0
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def round_bits(x, bits, least=0.0):
    """x at the nearest number of `bits` significant bits (a multiple of `least`), ties to even."""
    x = np.asarray(x, dtype=np.float64)
    _, e = np.frexp(x)
    step = np.maximum(np.ldexp(1.0, np.asarray(e) - bits), least)
    return np.round(x / step) * step


def scales(x, fmt):
    """x [..., groups, 32] -> the scale of each group, [..., groups]."""
    fine = np.where(np.isfinite(x), x, 0.0)
    hi, lo = fine.max(axis=-1), fine.min(axis=-1)
    d = np.where(hi >= -lo, hi, lo) / -8.0 if fmt == I4 else np.maximum(hi, -lo) / 6.0
    d = np.clip(d, -TOP_SCALE, TOP_SCALE)
    return round_bits(round_bits(d, 8), 11, 2.0 ** -24)


def values(rows, fmt):
    """What the cache holds of rows [..., head_dim]: code times scale."""
    x = np.asarray(rows, dtype=np.float64)
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // GROUP, GROUP))
    d = scales(g, fmt)[..., None]
    g = np.clip(np.where(np.isnan(g), 0.0, g), -1e300, 1e300)
    y = np.divide(g, d, out=np.zeros_like(g), where=d != 0)
    if fmt == I4:
        q = np.clip(np.round(y), -8, 7)
    else:
        mag = np.minimum(np.abs(y), 6.0)
        i = np.clip(np.searchsorted(GRID, mag, side="left"), 1, 7)   # GRID[i - 1] < mag <= GRID[i]
        mid = (GRID[i - 1] + GRID[i]) / 2
        up = (mag > mid) | ((mag == mid) & (i % 2 == 0))
        q = np.where(up, GRID[i], GRID[i - 1]) * np.sign(y)
    return (q * d).reshape(x.shape)


def attend(q, k, v, n_rows):
    """q [rows][Hq][hd], the last n_rows positions' queries over k, v [n][H][hd] -> (out, bound on its error).

    The bound counts roundings.  With A the largest sum_d |q_d k_d| / sqrt(hd) of a row and W = sum_j w_j |v_j|:
    - a score is off by at most A 2^-18.5: parts of q dropped (2^-22), 8 tensor-core steps that each cut 17 terms
      at 2^-24 of the running sum (2^-19.9 at most 2^-19.5 with the two halves' sum), its scaling and the
      subtraction of the maximum (2^-22); weights are off twice that (their own score's and the sum's);
    - ex2 and the dropped part of a weight 2^-21, 4 tensor-core steps 2^-20.9, dividing and joining 2^-21: 2^-19;
    - one fp32 rounding of the output and of the sum for each 64 positions: 2^-23 each;
    - a weight's two f16 parts end at f16's least step: each is off by at most 2^-25 where the largest weight stands at
      2^8 or above, so 2^-32 of the largest weight is lost of every position, however small its own is.
    """
    n_q, Hq, hd = q.shape
    n, H = k.shape[0], k.shape[1]
    G = Hq // H
    out = np.zeros((n_q, Hq, hd))
    bound = np.full((n_q, Hq, hd), 1e-30)
    for i in range(n_q):
        m = n - (n_rows - 1 - i)
        if m <= 0:
            continue
        for h in range(Hq):
            kk, vv = k[:m, h // G], v[:m, h // G]
            s = kk @ q[i, h] / math.sqrt(hd)
            w = np.exp(s - s.max())
            w /= w.sum()
            out[i, h] = w @ vv
            A = float((np.abs(kk) @ np.abs(q[i, h])).max() / math.sqrt(hd))
            W = w @ np.abs(vv)
            bound[i, h] += 2.0 ** -32 * w.max() * np.abs(vv).sum(axis=0) + W * (2 * A * 2.0 ** -18.5 + 2.0 ** -19 + (m / PAGE + 1) * 2.0 ** -23)
    return out, bound


def pages_step(table, held, keep, new, free, n_free, n_pages, n_tok):
    """One step of the tables (lists, changed in place) -> (n_free, q_start, slots, positions, wrong)."""
    R, W = len(held), len(table[0])
    npg = lambda n: -(-n // PAGE)  # noqa: E731
    wrong, plan = False, []
    for r in range(R):
        h, n = held[r], new[r]
        bad = h < 0 or h > W * PAGE
        h = 0 if bad else h
        k = h if keep is None else keep[r]
        bad = bad or k < 0 or k > h or n < 0 or k + max(n, 0) > W * PAGE
        plan.append([h, min(max(k, 0), h), max(n, 0), bad])
        wrong |= bad
    for r, (h, k, n, bad) in enumerate(plan):
        if not bad:
            for j in range(npg(k + n), npg(h)):
                free[n_free] = table[r][j]
                n_free += 1
    top, asked = n_free, 0
    q_start, slots, positions = [0], [], []
    for r, (h, k, n, bad) in enumerate(plan):
        need = 0 if bad else max(0, npg(k + n) - npg(h))
        asked += need
        refused = bad or (need > 0 and asked > top)
        wrong |= refused
        if not refused:
            for j in range(need):
                n_free -= 1
                table[r][npg(h) + j] = free[n_free]
            held[r] = k + n
        for p in range(k, k + min(n, n_tok + 1)):     # (rows behind n_tok need not all be listed)
            slots.append(-1 if refused else table[r][p // PAGE] * PAGE + p % PAGE)
            positions.append(p)
        q_start.append(len(slots))
    wrong |= len(slots) > n_tok
    slots, positions = slots[:n_tok], positions[:n_tok]
    pad = n_tok - len(slots)
    return n_free, [min(x, n_tok) for x in q_start], slots + [-1] * pad, positions + [0] * pad, wrong


def frequencies(rot, theta, scaling, factor=1.0, old_len=0.0, low=0.0, high=0.0, divisors=None):
    """w_i of the header's formulas, by names of the scaling."""
    u = np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)])
    s = factor
    if scaling == "linear":
        u = u / s
    elif scaling == "base":
        u = np.array([(theta * s ** (rot / (rot - 2.0))) ** (-2.0 * i / rot) for i in range(rot // 2)])
    elif scaling == "bands":
        low, high = low or 1.0, high or 4.0
        k = np.clip((old_len * u / (2 * math.pi) - low) / (high - low), 0, 1)
        u = u * k + u / s * (1 - k)
    elif scaling == "ramp":
        low, high = low or 1.0, high or 32.0
        pair = lambda t: rot * math.log(old_len / (2 * math.pi * t)) / (2 * math.log(theta))  # noqa: E731
        a, b = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot - 1)
        b = a + 0.001 if b <= a else b
        k = np.clip((np.arange(rot // 2) - a) / (b - a), 0, 1)
        u = u * (1 - k) + u / s * k
    return u if divisors is None else u / np.asarray(divisors, dtype=np.float64)


def rotate(x, positions, freq, layout, mag=1.0):
    """Rows x [n][heads][hd] turned at their positions: layout 0 adjacent pairs, 1 halves."""
    y = np.array(x, dtype=np.float64)
    half = len(freq)
    ang = np.asarray(positions, dtype=np.float64)[:, None] * freq
    c, s = mag * np.cos(ang)[:, None], mag * np.sin(ang)[:, None]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if layout == 0 else (slice(0, half), slice(half, 2 * half))
    u, v = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = u * c - v * s, u * s + v * c
    return y
