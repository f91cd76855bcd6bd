"""The 8-bit KV cache and its attentions in plain numpy, 64 bits: the oracle of
the GPU kernels (its own pins are in test_kv8_ref.py)."""
import math

import numpy as np

I8, E4M3 = 0, 1
B = 64
QMAX = {I8: 127.0, E4M3: 448.0}


def blocks(n):
    return (n + B - 1) // B


def scale_for(a, qmax):
    """The least power of two t >= 2^-100 with a <= qmax t."""
    e = -100
    if a > 0:
        e = max(e, math.frexp(a)[1] - math.frexp(qmax)[1] - 2)
        while a > qmax * 2.0 ** e:
            e += 1
    return 2.0 ** e


def _e4m3_table():
    t = np.empty(256)
    for b in range(256):
        s, e, m = b >> 7, (b >> 3) & 15, b & 7
        v = (1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6
        t[b] = -v if s else v
    return t


E4M3_VALUES = _e4m3_table()  # (0x7F and 0xFF are NaN in E4M3 and never written)


def to_values(b, fmt):
    return b.view(np.int8).astype(np.float64) if fmt == I8 else E4M3_VALUES[b]


def round8(x, fmt):
    """Values over the scale at the nearest 8-bit value, ties to even, saturating."""
    q = np.clip(x, -QMAX[fmt], QMAX[fmt])
    if fmt == I8:
        return np.rint(q)
    _, e = np.frexp(q)
    step = 2.0 ** (np.maximum(e - 1, -6) - 3.0)
    return np.rint(q / step) * step


def to_bytes(v, fmt):
    """8-bit values to their bytes (negative zero keeps its sign)."""
    if fmt == I8:
        return v.astype(np.int8).view(np.uint8)
    mag = np.abs(v)
    order = E4M3_VALUES[:127]
    b = np.searchsorted(order, mag).astype(np.uint8)
    assert np.array_equal(order[b], mag)
    return b | (np.signbit(v).astype(np.uint8) << 7)


class Cache:
    """State of one layer's cache, as bytes and scales."""

    def __init__(self, fmt, n_kvh, hd, stride):
        self.fmt, self.H, self.hd, self.stride = fmt, n_kvh, hd, stride
        nb = blocks(stride)
        self.data = {w: np.zeros((n_kvh, stride, hd), np.uint8) for w in "kv"}
        self.scale = {w: np.zeros((n_kvh, nb)) for w in "kv"}
        self.kmin = np.zeros((n_kvh, nb, hd), np.int8)
        self.kmax = np.zeros((n_kvh, nb, hd), np.int8)

    def append(self, k, v, pos):
        """k, v [n][H][hd], any float type."""
        n = k.shape[0]
        for w, src in (("k", k), ("v", v)):
            for h in range(self.H):
                x = src[:, h].astype(np.float64)
                b = pos // B
                while b * B < pos + n:
                    lo, hi = max(pos, b * B), min(pos + n, (b + 1) * B)
                    self._block(w, h, b, lo, hi, x[lo - pos:hi - pos])
                    b += 1

    def _block(self, w, h, b, lo, hi, x):
        fmt = self.fmt
        finite = np.abs(x)[np.isfinite(x)]
        t = scale_for(finite.max() if finite.size else 0.0, QMAX[fmt])
        if lo > b * B:
            old = self.scale[w][h, b]
            t = max(t, old)
            rows = slice(b * B, lo)
            q = round8(to_values(self.data[w][h, rows], fmt) * old / t, fmt)
            self.data[w][h, rows] = to_bytes(q, fmt)
        x = np.where(np.isnan(x), 0.0, x)
        self.data[w][h, lo:hi] = to_bytes(round8(x / t, fmt), fmt)
        self.scale[w][h, b] = t
        if w == "k":
            q = to_values(self.data[w][h, b * B:hi], fmt)
            u = 1.0 if fmt == I8 else 4.0
            self.kmin[h, b], self.kmax[h, b] = np.floor(q.min(axis=0) / u), np.ceil(q.max(axis=0) / u)

    def read(self, w, at):
        """Values of positions `at` (indices): [H][len][hd]."""
        at = np.asarray(at, dtype=np.int64)
        return to_values(self.data[w][:, at], self.fmt) * self.scale[w][:, at // B][..., None]


def attend(q, k, v, vs=None):
    """q [R][hd], k, v [n][hd], vs [n] the scales of v (None: ones) -> (out [R][hd], tolerance [R][hd]).

    The tolerance follows the kernel's arithmetic.  A score: q's two f16 parts
    carry 2^-22 of each product's size; the tensor cores add hd / 16 groups
    with at most 2^-22 of the summed sizes each; scaling and subtracting the
    maximum round three times.  A probability: the exponential 2^-21, its two f16
    parts 2^-22.  Sums over positions: at most one rounding of 2^-23 per step of
    16 positions a warp takes (n / 16 bounds them) and per merged partial (200).
    Underflow: the f16 operand of position i is p_i vs_i 2^8 / 2^m with 2^m at most the
    largest p_j 2^floor(log2 vs_j) (vs_j floored at 2^-64), and its low part is a
    multiple of f16's smallest step 2^-24: half of it, 2^-25, times 2^m / 2^8 and the
    cached value |v_i| / vs_i, for every position.  It is all that is left of a channel
    whose dominant positions hold an exact zero.
    """
    R, hd = q.shape
    if k.shape[0] == 0:
        return np.zeros_like(q), np.zeros_like(q)
    s = q @ k.T / math.sqrt(hd)
    size = np.abs(q) @ np.abs(k).T / math.sqrt(hd)
    m = s.max(axis=1, keepdims=True)
    p = np.exp(s - m)
    p /= p.sum(axis=1, keepdims=True)
    out = p @ v
    es = size.max(axis=1, keepdims=True) * (2.0 ** -22 * (hd / 16 + 2)) + 3 * 2.0 ** -24 * np.abs(s).max(
        axis=1, keepdims=True)
    rel = 2 * (es + 2.0 ** -21) + 2.0 ** -21 + (min(k.shape[0] / 16, 200) + 200) * 2.0 ** -23
    vs = np.ones(k.shape[0]) if vs is None else vs
    top = (p * np.maximum(vs, 2.0 ** -64)).max(axis=1, keepdims=True)
    cached = (np.abs(v) / np.where(vs == 0, 1.0, vs)[:, None]).sum(axis=0)
    return out, rel * (p @ np.abs(v)) + 2.0 ** -33 * top * cached + 1e-30


def attend_cache(c, q, n_pos, lists=None):
    """q [nq][n_qh][hd] -> (out, tolerance); lists [nq][H][n_sel]: blocks attended to (None: all)."""
    nq, n_qh, hd = q.shape
    G = n_qh // c.H
    out, tol = np.empty(q.shape), np.empty(q.shape)
    full = None
    if lists is None:
        at = np.arange(n_pos + nq - 1)
        full = c.read("k", at), c.read("v", at), c.scale["v"][:, at // B]
    for i in range(nq):
        n = n_pos + i
        for g in range(c.H):
            if lists is None:
                k, v, vs = (x[g, :n] for x in full)
            else:
                at = [np.arange(b * B, min(n, b * B + B)) for b in lists[i][g] if 0 <= b < blocks(n)]
                at = np.concatenate(at) if at else np.zeros(0, np.int64)
                k, v, vs = c.read("k", at)[g], c.read("v", at)[g], c.scale["v"][g, at // B]
            sl = slice(g * G, (g + 1) * G)
            out[i, sl], tol[i, sl] = attend(q[i, sl].astype(np.float64), k, v, vs)
    return out, tol


def select(c, q, n_pos, n_sel, n_first, n_last):
    nq, n_qh, hd = q.shape
    G = n_qh // c.H
    idx = np.full((nq, c.H, n_sel), -1, np.int32)
    for i in range(nq):
        nb = blocks(n_pos + i)
        for g in range(c.H):
            if nb <= n_sel:
                idx[i, g, :nb] = np.arange(nb)
                continue
            x = q[i, g * G:(g + 1) * G].astype(np.float64)
            finite = np.abs(x)[np.isfinite(x)]
            t = scale_for(finite.max() if finite.size else 0.0, 2047.0)
            qi = np.rint(np.clip(np.where(np.isnan(x), 0.0, x / t), -2047, 2047)).astype(np.int64)
            lo, hi = c.kmin[g, :nb].astype(np.int64), c.kmax[g, :nb].astype(np.int64)
            s = np.maximum(qi[:, None] * lo, qi[:, None] * hi).sum(axis=(0, 2))
            score = s.astype(np.float32).astype(np.float64) * c.scale["k"][g, :nb]
            forced = (np.arange(nb) < n_first) | (np.arange(nb) >= nb - n_last)
            order = sorted(range(nb), key=lambda b: (not forced[b], -score[b], b))
            idx[i, g] = sorted(order[:n_sel])
    return idx
