"""The oracle of kv8_ref at tolerances that follow the launch: how many partial
results a call of the attention merges is worked out from the shape, as the
launcher does, instead of bounded for every shape at once."""
import math

import numpy as np

import kv8_ref as ref

WARPS, MAX_CLUSTER, MAX_SPLITS = 8, 16, 512


def plan(sms, H, G, hd, nq, n_pos, n_sel=0):
    """The launch of nt_attn_kv8 (n_sel 0) or nt_attn_kv8_blocks with a host position: rows in eights R, 16-token
    units of a step U, splits S, whether they are one cluster, steps of the busiest warp."""
    sparse = n_sel > 0
    rows = G if sparse else G * nq
    R = 2 if rows > 8 else 1
    chunks = -(-rows // (8 * R))
    z = chunks * nq if sparse else chunks
    most = n_sel * ref.B if sparse else n_pos + nq - 1
    S = max(1, min(MAX_SPLITS, sms * (2 if R == 1 else 1) // (H * z)))
    useful = lambda u: max(1, -(-most // (16 * WARPS * u)))  # noqa: E731
    groups = H * z
    widest = min(MAX_CLUSTER, R * hd // 8, S, S if R == 1 else sms // 2 // groups)
    C = 1
    while C < useful(R) and 2 * C <= widest:
        C *= 2
    cluster = useful(2) > 1 and C > 1 and most <= 768 * C
    if cluster:
        S = C
    long_from = 640 * S if cluster else 32 * WARPS * S
    U = 2 if R == 2 or most <= 32 * WARPS or most >= long_from else 1
    if not cluster:
        S = min(S, useful(U))
    per = max(WARPS, -(-(-(-most // (16 * U))) // S))
    return dict(R=R, U=U, S=S, cluster=cluster, steps=-(-per // WARPS))


def attend(q, k, v, vs, p):
    """q [R][hd], k, v [n][hd], vs [n] the scales of v, p a plan -> (out, tolerance, rms of the error allowed / rms of out).

    Per element: a score carries q's two f16 parts (2^-22 of each product's size), at most 2^-22 of the summed
    sizes for each of hd / 16 k-steps of the tensor cores, and three fp32 roundings; a probability 2^-21 of the
    exponential and 2^-22 of its two f16 parts, once in the output and once in the sum; the sums take 2^-23 per
    step of a warp (twice: the sum and the output), per merged warp and split, and 8 more inside a step; what an
    f16 operand cannot hold is half of its smallest step, 2^-25, over 2^8 of the largest operand p vs.

    As an rms the roundings do not line up: a score is off by at most 2^-23 of the scores' rms per k-step, and the
    exponential, the f16 parts and the sums together by 2^-21.
    """
    R, hd = q.shape
    if k.shape[0] == 0:
        return np.zeros_like(q), np.zeros_like(q), 0.0
    s = q @ k.T / math.sqrt(hd)
    size = (np.abs(q) @ np.abs(k).T).max(axis=1, keepdims=True) / math.sqrt(hd)
    w = np.exp(s - s.max(axis=1, keepdims=True))
    w /= w.sum(axis=1, keepdims=True)
    out = w @ v
    es = size * (2.0 ** -22 * (hd / 16 + 1)) + 3 * 2.0 ** -24 * np.abs(s).max(axis=1, keepdims=True)
    rel = 2 * (es + 2.0 ** -21 + 2.0 ** -22) + (2 * p["steps"] + 2 * (WARPS + p["S"]) + 8) * 2.0 ** -23
    top = (w * vs).max(axis=1, keepdims=True)
    cached = (np.abs(v) / vs[:, None]).sum(axis=0)
    rms = math.sqrt(np.mean(s * s)) * hd / 16 * 2.0 ** -23 + 2.0 ** -21
    return out, rel * (w @ np.abs(v)) + 2.0 ** -33 * top * cached, rms


def check(got, c, q, n_pos, p, lists=None, rms=True):
    """got [nq][n_qh][hd] against the oracle cache c: every element, and the error of the whole."""
    nq, n_qh, hd = q.shape
    G = n_qh // c.H
    err2 = want2 = 0.0
    bar = 0.0
    for g in range(c.H):
        sl = slice(g * G, (g + 1) * G)
        if lists is None:
            at = np.arange(n_pos + nq - 1)
            full = [ref.to_values(c.data[w][g, at], c.fmt) * c.scale[w][g, at // ref.B][:, None] for w in "kv"]
        for i in range(nq):
            n = n_pos + i
            if lists is None:
                k, v, vs = full[0][:n], full[1][:n], c.scale["v"][g, at[:n] // ref.B]
            else:
                pos = [np.arange(b * ref.B, min(n, (b + 1) * ref.B)) for b in lists[i][g] if 0 <= b < ref.blocks(n)]
                pos = np.concatenate(pos) if pos else np.zeros(0, np.int64)
                k, v = (ref.to_values(c.data[w][g, pos], c.fmt) * c.scale[w][g, pos // ref.B][:, None] for w in "kv")
                vs = c.scale["v"][g, pos // ref.B]
            want, tol, r = attend(q[i, sl].astype(np.float64), k, v, vs, p)
            err = got[i, sl].astype(np.float64) - want
            assert np.all(np.abs(err) <= tol), (g, i, np.nanmax(np.abs(err) / tol), np.isnan(err).sum())
            err2, want2, bar = err2 + np.sum(err * err), want2 + np.sum(want * want), max(bar, r)
    if rms and want2:
        assert math.sqrt(err2 / want2) <= bar, (math.sqrt(err2 / want2), bar)
    return math.sqrt(err2 / want2) if want2 else 0.0
