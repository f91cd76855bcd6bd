"""The operators over the 8-bit KV cache, as they are timed and compared.

Three operators, in a plain form (elementary torch operations) and as calls of
the library:

- ``write``: rows of K and V quantised into the cache (``nt_kv8_append``) and
  the touched blocks read back (``nt_kv8_read``);
- ``attend``: grouped-query attention over the cache (``nt_attn_kv8``), one
  query for a decode step, several for the causal verify pass;
- ``sparse``: the blocks each query reads are chosen by a bound on their scores
  (``nt_kv8_select``), then attended to (``nt_attn_kv8_blocks``).

The cache holds K and V in 8 bits, ``[n_kvh][kv_stride][head_dim]``, with one
power-of-two scale for each block of 64 positions and head.  ``i8`` values are
q * t with |q| <= 127, ``e4m3`` values e4m3 numbers times t.  ``kmin`` and
``kmax`` hold each block's smallest and largest k of every channel, as integers
in units of t (i8) or 4 t (e4m3).
"""
import math

import torch

own = False

BLOCK = 64
QMAX = {"i8": 127.0, "e4m3": 448.0}
MIN_EXP = -100   # the least scale is 2^-100
QSEL = 2047.0    # the selection's queries are rounded to 12-bit integers


# ---- cases -----------------------------------------------------------------------
def listed():
    return [
        # one token of a Llama-8B-shaped decode step enters the cache (a block in the middle)
        dict(name="write_decode_i8", op="write", fmt="i8", n_kvh=8, hd=128, stride=1160, pos=1087, n=1, src="f32"),
        # a speculative verify pass writes 5 tokens across a block's end
        dict(name="write_verify_e4m3", op="write", fmt="e4m3", n_kvh=8, hd=128, stride=4168, pos=4158, n=5, src="f32"),
        # a prompt's K/V rows, starting inside a block and ending inside one
        dict(name="write_prompt_i8", op="write", fmt="i8", n_kvh=8, hd=128, stride=33001, pos=33, n=32767, src="f32"),
        # a long F16 cache turned into an 8-bit one, and read back as F16
        dict(name="write_convert_e4m3", op="write", fmt="e4m3", n_kvh=8, hd=128, stride=131072, pos=0, n=131072,
             src="f16"),
        # decode attention at the 8B workload's length: latency counts
        dict(name="attend_1088_i8", op="attend", fmt="i8", n_qh=32, n_kvh=8, hd=128, stride=1160, n_pos=1088, nq=1),
        # decode attention at the 70B workload's shape and length
        dict(name="attend_4160_e4m3", op="attend", fmt="e4m3", n_qh=64, n_kvh=8, hd=128, stride=4168, n_pos=4160,
             nq=1),
        # decode attention over a long context, ragged
        dict(name="attend_131071_i8", op="attend", fmt="i8", n_qh=32, n_kvh=8, hd=128, stride=131077, n_pos=131071,
             nq=1),
        # the verify pass of 8 tokens, causal among them
        dict(name="attend_verify8_e4m3", op="attend", fmt="e4m3", n_qh=32, n_kvh=8, hd=128, stride=16400, n_pos=16381,
             nq=8),
        # the longest context
        dict(name="attend_1000003_i8", op="attend", fmt="i8", n_qh=32, n_kvh=8, hd=128, stride=1000100,
             n_pos=1000003, nq=1),
        # sparse decode attention, short: 16 of 65 blocks
        dict(name="sparse_4160_i8", op="sparse", fmt="i8", n_qh=64, n_kvh=8, hd=128, stride=4168, n_pos=4160, nq=1,
             n_sel=16, n_first=1, n_last=2),
        # sparse verify pass of 5 tokens over a long context: 64 of 2048 blocks each
        dict(name="sparse_131071_nq5_e4m3", op="sparse", fmt="e4m3", n_qh=32, n_kvh=8, hd=128, stride=131077,
             n_pos=131071, nq=5, n_sel=64, n_first=1, n_last=4),
        # sparse decode attention over the longest context: 128 of 15626 blocks
        dict(name="sparse_1000003_i8", op="sparse", fmt="i8", n_qh=32, n_kvh=8, hd=128, stride=1000100,
             n_pos=1000003, nq=1, n_sel=128, n_first=1, n_last=4),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "attend", "sparse"])
    hd = rng.choice([64, 128, 128])
    n_kvh = rng.choice([1, 2, 3, 4, 8])
    case = dict(op=op, fmt=rng.choice(["i8", "e4m3"]), n_kvh=n_kvh, hd=hd)
    if op == "write":
        n = _log_int(rng, 1, 120000)
        pos = rng.randrange(0, 200)
        case.update(n=n, pos=pos, stride=n + pos + rng.randrange(0, 100), src=rng.choice(["f32", "f32", "f16"]))
        return case
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    nq = rng.choice([1, 1, 1, 2, 5, 8, 16])
    # longest when one query attends; the work of many queries stays below the largest case's
    n_pos = _log_int(rng, 1, max(1000, 900000 // (nq * max(1, G // 4))))
    case.update(n_qh=n_kvh * G, n_pos=n_pos, nq=nq, stride=n_pos + nq + rng.randrange(0, 100))
    if op == "sparse":
        first, last = rng.randrange(0, 3), rng.randrange(1, 5)
        case.update(n_sel=_log_int(rng, 8, 256), n_first=first, n_last=last)
    return case


def _nblocks(n):
    return (n + BLOCK - 1) // BLOCK


def work(case):
    H, hd = case["n_kvh"], case["hd"]
    if case["op"] == "write":
        n, pos = case["n"], case["pos"]
        o0 = pos % BLOCK
        wide = 4 if case["src"] == "f32" else 2
        blocks = _nblocks(o0 + n)
        rows = n + o0                                   # rows read back
        b = 2 * H * hd * (n * wide + o0 + n + rows * wide)  # source, old rows, 8-bit rows, values read back
        b += H * blocks * (2 * 4 + 2 * hd)              # scales and summaries
        return {"bytes": b, "flops": 2 * H * hd * (4 * n + rows)}
    nq, Hq = case["nq"], case["n_qh"]
    tokens = case["n_pos"] + nq - 1
    io = 2 * nq * Hq * hd * 4
    if case["op"] == "attend":
        b = 2 * H * tokens * hd + 2 * 4 * H * _nblocks(tokens) + io
        return {"bytes": b, "flops": 4 * nq * Hq * hd * case["n_pos"]}
    nb = _nblocks(tokens)
    sel = min(nb, case["n_sel"])
    b = H * nb * (2 * hd + 4) + io + nq * H * case["n_sel"] * 4
    b += 2 * H * min(nb, nq * sel) * (BLOCK * hd + 4)
    return {"bytes": b, "flops": 4 * nq * H * nb * hd + 4 * nq * Hq * hd * min(tokens, sel * BLOCK)}


# ---- the plain form ----------------------------------------------------------------
def _scale_for(a, qmax):
    """The least power of two t >= 2^MIN_EXP with a <= qmax * t."""
    mq, eq = math.frexp(qmax)
    m, e = torch.frexp(a)
    e = e - eq + (m > mq)
    e = torch.where(a > 0, e, torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)
    return torch.ldexp(torch.ones_like(a), e)


def _round8(x, fmt):
    """x (already divided by its scale) at the nearest 8-bit value, ties to even; stays floating point."""
    if fmt == "i8":
        return torch.round(x)
    _, e = torch.frexp(x)                      # |x| in [2^(e-1), 2^e): 3 mantissa bits below the leading one
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _bytes(v, fmt):
    return (v.to(torch.int8) if fmt == "i8" else v.to(torch.float8_e4m3fn)).view(torch.uint8)


def _values(b, fmt):
    return b.view(torch.int8 if fmt == "i8" else torch.float8_e4m3fn).float()


def _spread(s, n):
    """Block scales [..., nb] over the first n positions [..., n, 1]."""
    return s.repeat_interleave(BLOCK, dim=-1)[..., :n, None]


def _summary(v, fmt):
    """v [..., rows, hd] (values over the scale): the integer bounds of each channel."""
    lo, hi = v.amin(dim=-2), v.amax(dim=-2)
    if fmt == "e4m3":
        lo, hi = torch.floor(lo / 4), torch.ceil(hi / 4)
    return lo.to(torch.int8), hi.to(torch.int8)


def _write_rows(x, data, scale, pos, fmt):
    """x [H, n, hd] into rows pos.. of data [H, stride, hd]; returns the touched rows' values over their scales."""
    n = x.shape[1]
    b0, o0 = pos // BLOCK, pos % BLOCK
    nb = _nblocks(o0 + n)
    pad = nb * BLOCK - o0 - n
    blocks = torch.nn.functional.pad(x, (0, 0, o0, pad)).unflatten(1, (nb, BLOCK))
    t = _scale_for(blocks.abs().amax(dim=(2, 3)), QMAX[fmt])
    if o0:
        t_old = scale[:, b0].clone()
        t[:, 0] = torch.maximum(t[:, 0], t_old)
    v = _round8(blocks / t[:, :, None, None], fmt)
    if o0:
        old = _values(data[:, pos - o0:pos].contiguous(), fmt) * (t_old / t[:, 0])[:, None, None]
        v[:, 0, :o0] = _round8(old, fmt)
    rows = v.flatten(1, 2)[:, :o0 + n]
    data[:, pos - o0:pos + n] = _bytes(rows.contiguous(), fmt)
    scale[:, b0:b0 + nb] = t
    return rows, nb


def _plain_write(st):
    c, fmt, pos, n = st["case"], st["case"]["fmt"], st["case"]["pos"], st["case"]["n"]
    o0, b0 = pos % BLOCK, pos // BLOCK
    outs = []
    for which in "kv":
        x = st[which + "_src"].float()
        x = x.transpose(0, 1) if c["src"] == "f32" else x[:, pos:pos + n]
        rows, nb = _write_rows(x, st[which], st[which + "scale"], pos, fmt)
        if which == "k":
            full = (rows.shape[1] // BLOCK) * BLOCK
            if full:
                lo, hi = _summary(rows[:, :full].unflatten(1, (-1, BLOCK)), fmt)
                st["kmin"][:, b0:b0 + full // BLOCK], st["kmax"][:, b0:b0 + full // BLOCK] = lo, hi
            if full < rows.shape[1]:
                st["kmin"][:, b0 + nb - 1], st["kmax"][:, b0 + nb - 1] = _summary(rows[:, full:], fmt)
        back = _values(st[which][:, pos - o0:pos + n].contiguous(), fmt)
        back = back * _spread(st[which + "scale"][:, b0:b0 + nb], o0 + n)
        outs.append(back if c["src"] == "f32" else back.half())
    return outs + [st["kscale"], st["vscale"], st["kmin"], st["kmax"]]


def _softmax_out(q, k, v, live, dtype):
    """q [R, hd], k, v [n, hd], live [R, n] bool: softmax(q.k / sqrt(hd)) v, zero for a row with nothing live."""
    if k.shape[0] == 0:
        return torch.zeros_like(q)
    s = (q @ k.T) / math.sqrt(q.shape[1])
    s = torch.where(live, s, torch.full((), -math.inf, dtype=dtype, device=s.device))
    m = s.amax(dim=1, keepdim=True)
    p = torch.where(live, torch.exp(s - m), torch.zeros((), dtype=dtype, device=s.device))
    total = p.sum(dim=1, keepdim=True)
    return torch.where(total > 0, (p @ v) / total, torch.zeros((), dtype=dtype, device=s.device))


def _plain_attend(st):
    c = st["case"]
    H, G, hd, nq, fmt = c["n_kvh"], c["n_qh"] // c["n_kvh"], c["hd"], c["nq"], c["fmt"]
    tokens = c["n_pos"] + nq - 1
    out = torch.empty(nq, H, G, hd, device="cuda")
    q = st["q"].view(nq, H, G, hd)
    limit = c["n_pos"] + torch.arange(nq, device="cuda").repeat_interleave(G)
    live = torch.arange(tokens, device="cuda")[None, :] < limit[:, None]
    for g in range(H):
        k = _values(st["k"][g, :tokens], fmt) * _spread(st["kscale"][g], tokens)
        v = _values(st["v"][g, :tokens], fmt) * _spread(st["vscale"][g], tokens)
        out[:, g] = _softmax_out(q[:, g].reshape(nq * G, hd), k, v, live, torch.float32).view(nq, G, hd)
    return out.view(nq, H * G, hd)


def _choose(score, nb, c):
    """Ascending indices of the chosen blocks among score[:nb], padded with -1 to n_sel."""
    idx = torch.full((c["n_sel"],), -1, dtype=torch.int32, device=score.device)
    if nb <= c["n_sel"]:
        idx[:nb] = torch.arange(nb, dtype=torch.int32, device=score.device)
        return idx
    s = score[:nb].clone()
    s[:c["n_first"]] = math.inf
    s[nb - c["n_last"]:] = math.inf
    order = torch.sort(s, descending=True, stable=True).indices[:c["n_sel"]]
    idx[:] = torch.sort(order).values.to(torch.int32)
    return idx


def _plain_sparse(st):
    c = st["case"]
    H, G, hd, nq, fmt = c["n_kvh"], c["n_qh"] // c["n_kvh"], c["hd"], c["nq"], c["fmt"]
    nb_all = _nblocks(c["n_pos"] + nq - 1)
    q = st["q"].view(nq, H, G, hd)
    tq = _scale_for(q.abs().amax(dim=(2, 3)), QSEL)
    qi = torch.round(q / tq[:, :, None, None]).double()
    # 64 bits: the sums are whole numbers above 2^24
    qp, qn = qi.clamp(min=0).sum(dim=2), qi.clamp(max=0).sum(dim=2)       # [nq, H, hd]
    hi, lo = st["kmax"][:, :nb_all].double(), st["kmin"][:, :nb_all].double()
    S = torch.einsum("ihd,hbd->ihb", qp, hi) + torch.einsum("ihd,hbd->ihb", qn, lo)
    score = S.float() * st["kscale"][None, :, :nb_all]
    idx = torch.empty(nq, H, c["n_sel"], dtype=torch.int32, device="cuda")
    out = torch.empty(nq, H, G, hd, device="cuda")
    within = torch.arange(BLOCK, device="cuda")
    for i in range(nq):
        limit = c["n_pos"] + i
        for g in range(H):
            idx[i, g] = _choose(score[i, g], _nblocks(limit), c)
            blocks = idx[i, g][:min(_nblocks(limit), c["n_sel"])].long()
            at = (blocks[:, None] * BLOCK + within).flatten()
            live = (at < limit)[None, :].expand(G, -1)
            at = at.clamp(max=limit - 1)
            k = _values(st["k"][g][at], fmt) * st["kscale"][g][at // BLOCK][:, None]
            v = _values(st["v"][g][at], fmt) * st["vscale"][g][at // BLOCK][:, None]
            out[i, g] = _softmax_out(q[i, g], k, v, live, torch.float32)
    return [idx, out.view(nq, H * G, hd)]


# ---- inputs -----------------------------------------------------------------------
def _rows(gen, n, hd, spread):
    """n rows of one head: channels of unequal size around slowly moving means, as keys have them."""
    size = torch.exp(spread * torch.randn(hd, generator=gen, device="cuda"))
    nb = _nblocks(n)
    drift = torch.randn(nb, hd, generator=gen, device="cuda").repeat_interleave(BLOCK, dim=0)[:n]
    return (torch.randn(n, hd, generator=gen, device="cuda") + 0.7 * drift) * size


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    H, hd, stride, fmt = case["n_kvh"], case["hd"], case["stride"], case["fmt"]
    nb = _nblocks(stride)
    st = {"case": case}
    for w in "kv":
        st[w] = torch.zeros(H, stride, hd, dtype=torch.uint8, device="cuda")
        st[w + "scale"] = torch.ones(H, nb, device="cuda")
    st["kmin"] = torch.zeros(H, nb, hd, dtype=torch.int8, device="cuda")
    st["kmax"] = torch.zeros(H, nb, hd, dtype=torch.int8, device="cuda")
    filled = case["pos"] if case["op"] == "write" else case["n_pos"] + case["nq"] - 1
    for g in range(H):
        for w, spread in (("k", 0.5), ("v", 0.2)):
            if not filled:
                continue
            rows, _ = _write_rows(_rows(gen, filled, hd, spread)[None], st[w][g:g + 1], st[w + "scale"][g:g + 1], 0,
                                  fmt)
            if w == "k":
                for b0, b1 in ((0, filled // BLOCK), (filled // BLOCK, _nblocks(filled))):
                    part = rows[0, b0 * BLOCK:b1 * BLOCK]
                    if b1 > b0:
                        lo, hi = _summary(part.unflatten(0, (b1 - b0, -1)), fmt)
                        st["kmin"][g, b0:b1], st["kmax"][g, b0:b1] = lo, hi
    if case["op"] == "write":
        n, pos = case["n"], case["pos"]
        for w, spread in (("k", 0.5), ("v", 0.2)):
            if case["src"] == "f32":   # the layout of a step's K or V rows: [token][head][hd]
                src = torch.empty(n, H, hd, device="cuda")
                for g in range(H):
                    src[:, g] = 1.5 * _rows(gen, n, hd, spread)
            else:                      # the layout of an F16 cache: [head][position][hd]
                src = torch.zeros(H, stride, hd, dtype=torch.float16, device="cuda")
                for g in range(H):
                    src[g, pos:pos + n] = 1.5 * _rows(gen, n, hd, spread)
            st[w + "_src"] = src
    else:
        st["q"] = torch.randn(case["nq"], case["n_qh"], hd, generator=gen, device="cuda") * 1.5
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if not own:
        return st
    from block_quantized_gemv_nt_gb300 import engine, nt
    fmt = nt.KV8_I8 if case["fmt"] == "i8" else nt.KV8_E4M3
    st["ctx"] = nt.Context(torch.cuda.current_device())
    cache = engine.KV8Cache(st["ctx"], fmt, case["n_kvh"], case["hd"], case["stride"],
                            buffers={n: st[n] for n in ("k", "v", "kscale", "vscale", "kmin", "kmax")})
    st["cache"] = cache
    if case["op"] == "write":
        rows = case["pos"] % BLOCK + case["n"]
        dt = torch.float32 if case["src"] == "f32" else torch.float16
        st["k_out"] = torch.empty(case["n_kvh"], rows, case["hd"], dtype=dt, device="cuda")
        st["v_out"] = torch.empty_like(st["k_out"])
    else:
        st["out"] = torch.empty_like(st["q"])
        if case["op"] == "sparse":
            st["idx"] = torch.empty(case["nq"], case["n_kvh"], case["n_sel"], dtype=torch.int32, device="cuda")
    return st


def run(st):
    c = st["case"]
    if not own:
        return {"write": _plain_write, "attend": _plain_attend, "sparse": _plain_sparse}[c["op"]](st)
    cache = st["cache"]
    if c["op"] == "write":
        pos, n = c["pos"], c["n"]
        if c["src"] == "f32":
            cache.append(st["k_src"], st["v_src"], pos)
        else:
            cache.append_from_heads(st["k_src"][:, pos:pos + n], st["v_src"][:, pos:pos + n], pos)
        cache.read(pos - pos % BLOCK, st["k_out"], st["v_out"])
        return [st["k_out"], st["v_out"], st["kscale"], st["vscale"], st["kmin"], st["kmax"]]
    if c["op"] == "attend":
        cache.attend(st["q"], st["out"], c["n_pos"])
        return st["out"]
    cache.select(st["q"], st["idx"], c["n_pos"], n_first=c["n_first"], n_last=c["n_last"])
    cache.attend_blocks(st["q"], st["out"], c["n_pos"], st["idx"])
    return [st["idx"], st["out"]]


# ---- the definition in 64 bits --------------------------------------------------------
def _exact_values(bits, fmt):
    """The number each byte stands for, from its bits."""
    b = bits.to(torch.int64)
    if fmt == "i8":
        return torch.where(b >= 128, b - 256, b).double()
    sign, e, m = b >> 7, (b >> 3) & 15, b & 7
    mag = torch.where(e > 0, (8 + m).double() * torch.exp2((e - 10).double()), m.double() * 2.0 ** -9)
    return torch.where(sign > 0, -mag, mag)


def _exact_round(x, fmt):
    """Nearest representable value by its distance to the grid, the even neighbour on a tie."""
    if fmt == "i8":
        grid = torch.ones_like(x)
    else:
        mag = x.abs().clamp(min=2.0 ** -6)
        e = torch.floor(torch.log2(mag))
        e = torch.where(torch.exp2(e) > mag, e - 1, torch.where(torch.exp2(e + 1) <= mag, e + 1, e))
        grid = torch.exp2(e - 3)
    lo = torch.floor(x / grid)
    up = x / grid - lo
    odd = torch.remainder(lo, 2) == 1
    return (lo + ((up > 0.5) | ((up == 0.5) & odd)).double()) * grid


def _exact_scale(a, qmax):
    t = torch.full_like(a, 2.0 ** MIN_EXP)
    e = torch.ceil(torch.log2((a / qmax).clamp(min=2.0 ** MIN_EXP)))
    for d in (-1, 0, 1):                      # the logarithm may be off by its last bit
        cand = torch.exp2(e + d).clamp(min=2.0 ** MIN_EXP)
        t = torch.where(((a > qmax * t) & (a <= qmax * cand)), cand, t)
    return t


def _exact_write(st):
    c = st["case"]
    fmt, pos, n, H, hd = c["fmt"], c["pos"], c["n"], c["n_kvh"], c["hd"]
    first, end = pos // BLOCK, _nblocks(pos + n)
    back = {}
    kmin, kmax = st["kmin"].clone(), st["kmax"].clone()
    scales = {w: st[w + "scale"].double() for w in "kv"}
    out_dt = torch.float32 if c["src"] == "f32" else torch.float16
    for w in "kv":
        back[w] = torch.empty(H, pos + n - first * BLOCK, hd, dtype=torch.float64, device="cuda")
        for g in range(H):
            src = (st[w + "_src"][:, g] if c["src"] == "f32" else st[w + "_src"][g, pos:pos + n]).double()
            row0 = first * BLOCK
            x = torch.zeros((end - first) * BLOCK, hd, dtype=torch.float64, device="cuda")
            x[pos - row0:pos + n - row0] = src
            x = x.view(end - first, BLOCK, hd)
            t = _exact_scale(x.abs().amax(dim=(1, 2)), QMAX[fmt])
            if pos > row0:
                t_old = scales[w][g, first].clone()
                t[0] = torch.maximum(t[0], t_old)
                x[0, :pos - row0] = _exact_values(st[w][g, row0:pos], fmt) * t_old
            val = _exact_round(x / t[:, None, None], fmt)
            scales[w][g, first:end] = t
            back[w][g] = (val * t[:, None, None]).view(-1, hd)[:pos + n - row0]
            if w == "k":
                unit = 1.0 if fmt == "i8" else 4.0
                rows = torch.arange((end - first) * BLOCK, device="cuda").view(end - first, BLOCK, 1) < pos + n - row0
                lo = torch.where(rows, val, math.inf).amin(dim=1)
                hi = torch.where(rows, val, -math.inf).amax(dim=1)
                kmin[g, first:end] = torch.floor(lo / unit).to(torch.int8)
                kmax[g, first:end] = torch.ceil(hi / unit).to(torch.int8)
    return [back["k"], back["v"], scales["k"], scales["v"], kmin, kmax]


def _exact_head(st, g, at):
    """K and V values of head g at the positions `at` (a slice or indices), with their block scales."""
    c = st["case"]
    k, v = _exact_values(st["k"][g][at], c["fmt"]), _exact_values(st["v"][g][at], c["fmt"])
    block = torch.arange(c["stride"], device="cuda")[at] // BLOCK
    return k * st["kscale"][g].double()[block][:, None], v * st["vscale"][g].double()[block][:, None]


def _exact_attend(st):
    c = st["case"]
    H, G, hd, nq = c["n_kvh"], c["n_qh"] // c["n_kvh"], c["hd"], c["nq"]
    q = st["q"].double().view(nq, H, G, hd)
    out = torch.empty_like(q)
    for g in range(H):
        k, v = _exact_head(st, g, slice(0, c["n_pos"] + nq - 1))
        for i in range(nq):
            n = c["n_pos"] + i
            p = torch.softmax(q[i, g] @ k[:n].T / math.sqrt(hd), dim=1)
            out[i, g] = p @ v[:n]
    return out.view(nq, H * G, hd)


def _exact_sparse(st):
    c = st["case"]
    H, G, hd, nq = c["n_kvh"], c["n_qh"] // c["n_kvh"], c["hd"], c["nq"]
    q = st["q"].double().view(nq, H, G, hd)
    out = torch.empty_like(q)
    idx = torch.full((nq, H, c["n_sel"]), -1, dtype=torch.int32, device="cuda")
    for i in range(nq):
        n = c["n_pos"] + i
        nb = _nblocks(n)
        for g in range(H):
            if nb > c["n_sel"]:
                qi = _exact_round(q[i, g] / _exact_scale(q[i, g].abs().amax(), QSEL), "i8")
                bound = torch.zeros(nb, dtype=torch.float64, device="cuda")
                for h in range(G):
                    pos = qi[h] > 0
                    side = torch.where(pos, st["kmax"][g, :nb].double(), st["kmin"][g, :nb].double())
                    bound += side @ qi[h]
                score = (bound.float().double() * st["kscale"][g, :nb].double()).cpu().tolist()
                forced = set(range(c["n_first"])) | set(range(nb - c["n_last"], nb))
                order = sorted(range(nb), key=lambda b: (b not in forced, -score[b], b))
                chosen = sorted(order[:c["n_sel"]])
            else:
                chosen = list(range(nb))
            idx[i, g, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
            at = torch.cat([torch.arange(b * BLOCK, min(n, (b + 1) * BLOCK)) for b in chosen]).cuda()
            k, v = _exact_head(st, g, at)
            out[i, g] = torch.softmax(q[i, g] @ k.T / math.sqrt(hd), dim=1) @ v
    return [idx, out.view(nq, H * G, hd)]


def exact(case, seed):
    st = _inputs(case, seed)
    return {"write": _exact_write, "attend": _exact_attend, "sparse": _exact_sparse}[case["op"]](st)
