"""The operators of a step of several requests over a paged 4-bit KV cache, as
they are timed and compared.

Four operators, in a plain form (elementary torch operations) and as calls of
the library:

- ``pages``: the requests' block tables grow and shrink to new lengths, and the
  new tokens get their slots and positions (``nt_kv4_pages``);
- ``rope``: rotary positions on the rows of q and k (``nt_rope_rows``), pairs
  interleaved or in halves, of a part of the head, scaled for long contexts;
- ``write``: rows of K and V quantised into their slots (``nt_kv4_append``) and
  read back (``nt_kv4_read``);
- ``attend``: grouped-query attention of each request's rows over its own pages
  (``nt_attn_kv4``), causal among the rows of a request.

The cache holds pages of 64 positions.  Every 32 channels of a row share a scale,
an f16 number of at most 8 significant bits: the nearest to x / -8 of the value x
of the largest magnitude (the positive one of two that tie) for ``i4`` (codes
-8 .. 7), to max|x| / 6 for ``e2m1`` (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6).
"""
import math
import random

import torch

own = False

PAGE = 64
GROUP = 32
PART = 1024
TOP_SCALE = 2720.0  # the largest scale, 170 * 2^4


# ---- cases -----------------------------------------------------------------------
def listed():
    return [
        # a decode step of 16 requests, the most that one pass of the weights takes: latency counts
        dict(name="pages_decode_16", op="pages", n_req=16, width=64, mean=1900, kind="decode"),
        # a server's step: requests that decode, verify drafts, start with a prompt, or end
        dict(name="pages_mixed_250", op="pages", n_req=250, width=1024, mean=6000, kind="mixed"),
        # the largest batch, most requests starting with their prompts
        dict(name="pages_prompts_1024", op="pages", n_req=1024, width=512, mean=900, kind="prompts"),
        # the q and k rows of 16 requests' decode step, adjacent pairs as the framework's models have them
        dict(name="rope_decode_16", op="rope", n_tok=16, n_qh=32, n_kvh=8, hd=128, rot=128, layout="pairs",
             scaling="none", dtype="f32", far=4000),
        # a prompt's rows, pairs in halves, frequencies scaled by bands
        dict(name="rope_prompt_halves", op="rope", n_tok=16381, n_qh=32, n_kvh=8, hd=128, rot=128, layout="halves",
             scaling="bands", dtype="f32", far=131000),
        # F16 rows far into a long context, three quarters of the head turned
        dict(name="rope_far_f16", op="rope", n_tok=8191, n_qh=64, n_kvh=8, hd=128, rot=96, layout="halves",
             scaling="ramp", dtype="f16", far=1000000),
        # one token of each of 16 requests
        dict(name="write_decode_16_i4", op="write", fmt="i4", n_kvh=8, hd=128, n_tok=16, src="f32", kind="decode"),
        # a prompt's rows
        dict(name="write_prompt_e2m1", op="write", fmt="e2m1", n_kvh=8, hd=128, n_tok=32767, src="f32", kind="prompt"),
        # an F16 cache's rows turned into a 4-bit one
        dict(name="write_convert_i4", op="write", fmt="i4", n_kvh=8, hd=128, n_tok=131072, src="f16", kind="prompt"),
        # one request at the 8B workload's length: latency counts
        dict(name="attend_1x1088_i4", op="attend", fmt="i4", n_qh=32, n_kvh=8, hd=128, n_req=1, longest=1088, nq=1),
        # 16 requests of unequal lengths at the 70B workload's shape, drafts being verified
        dict(name="attend_16_ragged_e2m1", op="attend", fmt="e2m1", n_qh=64, n_kvh=8, hd=128, n_req=16, longest=16381,
             nq=5),
        # the longest context
        dict(name="attend_1x1000003_i4", op="attend", fmt="i4", n_qh=32, n_kvh=8, hd=128, n_req=1, longest=1000003,
             nq=1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pages", "rope", "write", "attend", "attend"])
    if op == "pages":
        n_req = _log_int(rng, 1, 1024)
        return dict(op=op, n_req=n_req, width=_log_int(rng, 32, 512), mean=_log_int(rng, 20, min(6000, max(40, 500000 // n_req))),
                    kind=rng.choice(["decode", "mixed", "prompts"]))
    hd, n_kvh = rng.choice([64, 128, 128]), rng.choice([1, 2, 3, 4, 8])
    if op == "rope":
        return dict(op=op, n_tok=_log_int(rng, 1, 16000), n_qh=n_kvh * rng.choice([1, 2, 4]), n_kvh=n_kvh, hd=hd,
                    rot=rng.choice([hd, hd, hd // 2, hd // 4, hd - 8]), layout=rng.choice(["pairs", "halves"]),
                    scaling=rng.choice(["none", "linear", "base", "bands", "ramp"]),
                    dtype=rng.choice(["f32", "f32", "f16"]), far=_log_int(rng, 100, 1000000))
    if op == "write":
        return dict(op=op, fmt=rng.choice(["i4", "e2m1"]), n_kvh=n_kvh, hd=hd, n_tok=_log_int(rng, 1, 100000),
                    src=rng.choice(["f32", "f32", "f16"]), kind=rng.choice(["decode", "prompt"]))
    group, n_req = rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), _log_int(rng, 1, 64)
    nq = rng.choice([1, 1, 1, 2, 5, 8])
    # the work of many rows stays below the longest case's
    return dict(op=op, fmt=rng.choice(["i4", "e2m1"]), n_qh=n_kvh * group, n_kvh=n_kvh, hd=hd, n_req=n_req, nq=nq,
                longest=_log_int(rng, 1, max(200, 500000 // (n_req * nq * max(1, group // 4)))))


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _lengths(case, seed):
    """Host lengths of an attention case: (positions each request holds, rows each has), in an order by the seed."""
    rng = random.Random(7)
    n, longest, nq = case["n_req"], case["longest"], case["nq"]
    held = [longest] + [_log_int(rng, max(1, longest // 50), longest) for _ in range(n - 1)]
    rows = [nq] + [rng.randint(1, nq) for _ in range(n - 1)]
    if n > 2:
        rows[n // 2] = 0            # a slot of the batch that nobody uses
        held[n // 2] = 0
    order = random.Random(seed).sample(range(n), n)
    return [held[i] for i in order], [rows[i] for i in order]


def _requests(case, seed):
    """Host lengths of a tables case: (held, keep, new) of each request, within the table's width, in an order by the seed."""
    rng = random.Random(11)
    cap = case["width"] * PAGE
    held, keep, new = [], [], []
    for _ in range(case["n_req"]):
        h = min(_log_int(rng, max(1, case["mean"] // 8), case["mean"] * 2), cap - 40)
        kind = case["kind"] if case["kind"] != "mixed" else rng.choice(
            ["decode", "decode", "decode", "verify", "prompts", "end", "idle"])
        if kind == "prompts" and rng.random() < 0.9:
            h, k, n = 0, 0, min(_log_int(rng, max(1, case["mean"] // 8), case["mean"] * 2), cap)
        elif kind == "verify":
            k = max(0, h - rng.randint(0, 4))
            n = 5
        elif kind == "end":
            k, n = 0, 0
        elif kind == "idle":
            k, n = h, 0
        else:
            k, n = h, 1
        held.append(h), keep.append(k), new.append(n)
    order = random.Random(seed).sample(range(len(held)), len(held))
    return [held[i] for i in order], [keep[i] for i in order], [new[i] for i in order]


def work(case):
    op = case["op"]
    if op == "pages":
        held, keep, new = _requests(case, 0)
        tok = sum(new)
        moved = sum(abs(_pages(k + n) - _pages(h)) for h, k, n in zip(held, keep, new))
        return {"bytes": case["n_req"] * 4 * 5 + 12 * tok + 8 * moved + 4 * sum(_pages(k % PAGE + n) for k, n in zip(keep, new)),
                "flops": case["n_req"] * 8 + 4 * tok}
    if op == "rope":
        wide = 4 if case["dtype"] == "f32" else 2
        rows = case["n_tok"] * (case["n_qh"] + case["n_kvh"])
        return {"bytes": 2 * rows * case["hd"] * wide + 4 * case["n_tok"], "flops": 3 * rows * case["rot"]}
    hd, H = case["hd"], case["n_kvh"]
    cell = hd // 2 + 2 * (hd // GROUP)      # bytes of one row of K or V in the cache
    if op == "write":
        wide = 4 if case["src"] == "f32" else 2
        return {"bytes": 2 * H * case["n_tok"] * (2 * hd * wide + 2 * cell) + 16 * case["n_tok"],
                "flops": 2 * H * hd * 5 * case["n_tok"]}
    held, rows = _lengths(case, 0)
    tok = sum(rows)
    return {"bytes": 2 * H * cell * sum(held) + 8 * tok * case["n_qh"] * hd + 4 * sum(_pages(h) for h in held),
            "flops": 4 * case["n_qh"] * hd * sum(h * r for h, r in zip(held, rows))}


# ---- the plain form ----------------------------------------------------------------
def _plain_pages(st):
    held, keep, new, table = st["held"].long(), st["keep"].long(), st["new"].long(), st["table"].long()
    n_tok, (R, W), P = st["n_tok"], table.shape, st["free"].numel()
    dev = table.device
    col = torch.arange(W, device=dev)[None, :]
    have, want = (held + PAGE - 1) // PAGE, (keep + new + PAGE - 1) // PAGE
    back, need = (have - want).clamp(min=0), (want - have).clamp(min=0)
    # pages given back go onto the stack in the order of the requests
    at = st["n_free"].long() + (back.cumsum(0) - back)[:, None] + col - want[:, None]
    given = (col >= want[:, None]) & (col < have[:, None])
    stack = torch.cat([st["free"].long(), torch.zeros(1, dtype=torch.long, device=dev)])
    stack = stack.scatter(0, torch.where(given, at, P).flatten(), torch.where(given, table, 0).flatten())
    top = st["n_free"].long() + back.sum()
    total = need.cumsum(0)
    ok = (need == 0) | (total <= top)
    at = top - 1 - (total - need)[:, None] - (col - have[:, None])
    taken = (col >= have[:, None]) & (col < want[:, None]) & ok[:, None]
    table = torch.where(taken, stack[at.clamp(0, P - 1)], table)
    q_start = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), new.cumsum(0)])
    i = torch.arange(n_tok, device=dev)
    r = torch.searchsorted(q_start[1:], i, right=True)
    pos = keep[r] + i - q_start[r]
    slots = torch.where(ok[r], table[r, pos // PAGE] * PAGE + pos % PAGE, -1)
    return {"table": table.int(), "free": stack[:P].int(), "n_free": (top - (need * ok).sum()).int(),
            "held": torch.where(ok, keep + new, held).int(), "q_start": q_start.int(), "slots": slots,
            "positions": pos.int()}


def _plain_rope_rows(x, cos, sin, case):
    rot, half = case["rot"], case["rot"] // 2
    part = x[..., :rot].float()
    if case["layout"] == "pairs":
        a, b = part[..., 0::2], part[..., 1::2]
    else:
        a, b = part[..., :half], part[..., half:]
    c, s = cos[:, None], sin[:, None]
    u, v = a * c - b * s, a * s + b * c
    turned = torch.stack([u, v], dim=-1).flatten(-2) if case["layout"] == "pairs" else torch.cat([u, v], dim=-1)
    return torch.cat([turned.to(x.dtype), x[..., rot:]], dim=-1)


def _plain_rope(st):
    # 64 bits: angles of far positions
    angle = st["positions"].double()[:, None] * st["freq"]
    cos, sin = (torch.cos(angle) * st["mag"]).float(), (torch.sin(angle) * st["mag"]).float()
    return [_plain_rope_rows(st[w], cos, sin, st["case"]) for w in ("q", "k")]


def _scale8(d):
    """d (64 bits) at the nearest f16 number of at most 8 significant bits, ties to even."""
    d = d.clamp(-TOP_SCALE, TOP_SCALE)
    step = ((torch.frexp(d).exponent.long() - 8 + 1023) << 52).view(torch.float64)  # a power of two, from its bits
    return (torch.round(d / step) * step).half()


def _quantise(x, fmt):
    """x [..., hd] -> (codes 0 .. 15 as uint8, scales f16 [..., hd / 32])."""
    g = x.float().unflatten(-1, (-1, GROUP))
    # 64 bits from here: quotients next to the border between two codes
    if fmt == "i4":
        hi, lo = g.amax(dim=-1, keepdim=True), g.amin(dim=-1, keepdim=True)
        d = _scale8(torch.where(hi >= -lo, hi, lo).double() / -8.0)
        q = torch.where(d == 0, 0.0, torch.round(g.double() / d.double())).clamp(-8, 7)
        code = (q + 8).to(torch.uint8)
    else:
        mag = g.abs()
        d = _scale8(mag.amax(dim=-1, keepdim=True).double() / 6.0)
        y = torch.where(d == 0, 0.0, mag.double() / d.double())
        code = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
        code = (code + 8 * (g < 0)).to(torch.uint8)
    return code.flatten(-2), d[..., 0]


def _values(code, scale, fmt):
    """The numbers that codes [..., hd] with scales [..., hd / 32] stand for, fp32 (exact)."""
    if fmt == "i4":
        v = code.float() - 8.0
    else:
        v = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                         device=code.device)[code.int()]
    return (v.unflatten(-1, (-1, GROUP)) * scale.float()[..., None]).flatten(-2)


def _pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _unpack(b):
    return torch.stack([b & 15, b >> 4], dim=-1).flatten(-2)


def _plain_write(st):
    fmt, slots = st["case"]["fmt"], st["slots"]
    outs = []
    for w in "kv":
        code, scale = _quantise(st[w + "_src"], fmt)
        st[w][slots], st[w + "scale"][slots] = _pack(code), scale
        outs.append(_values(_unpack(st[w][slots]), st[w + "scale"][slots], fmt).to(st[w + "_src"].dtype))
    return outs


def _plain_attend(st):
    c = st["case"]
    H, G, hd, fmt = c["n_kvh"], c["n_qh"] // c["n_kvh"], c["hd"], c["fmt"]
    R, NQ, n_tok = c["n_req"], c["nq"], st["q"].shape[0]
    n = -(-c["longest"] // PART) * PART
    dev = st["q"].device
    col = torch.arange(n, device=dev)
    at = st["table"].long()[:, (col // PAGE).clamp(max=st["table"].shape[1] - 1)] * PAGE + col % PAGE
    k, v = (_values(_unpack(st[w][at]), st[w + "scale"][at], fmt).transpose(1, 2) for w in "kv")   # [R, H, n, hd]
    first, rows = st["q_start"][:-1].long(), (st["q_start"][1:] - st["q_start"][:-1]).long()
    i = torch.arange(NQ, device=dev)
    q = st["q"][(first[:, None] + i).clamp(max=n_tok - 1)].view(R, NQ, H, G, hd).transpose(1, 2).reshape(R, H, NQ * G, hd)
    limit = (st["held"].long() - rows)[:, None] + 1 + i                                             # [R, NQ]
    live = (torch.arange(n, device=dev) < limit.repeat_interleave(G, dim=1)[:, :, None])[:, None]
    s = torch.where(live, (q @ k.transpose(2, 3)) / math.sqrt(hd), -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    p = torch.where(live, torch.exp(s - m), 0.0)
    # the sums of PART positions each are added in 64 bits: a long sum loses what its terms cancel to
    total = p.double().sum(dim=-1, keepdim=True)
    pv = (p.unflatten(3, (-1, PART)).transpose(2, 3) @ v.unflatten(2, (-1, PART))).double().sum(dim=2)
    out = torch.where(total > 0, pv / total, 0.0).float().view(R, H, NQ, G, hd).transpose(1, 2).reshape(R, NQ, H * G, hd)
    t = torch.arange(n_tok, device=dev)
    r = torch.searchsorted(st["q_start"][1:].long(), t, right=True)
    return out[r, t - first[r]]


# ---- inputs -----------------------------------------------------------------------
def _frequencies(case):
    """Host frequencies of the pairs (radians a position) and the magnitude of the turned channels."""
    rot, theta, factor, old = case["rot"], 500000.0, 8.0, 8192.0
    half = rot // 2
    w = [theta ** (-2.0 * i / rot) for i in range(half)]
    if case["scaling"] == "linear":
        return [x / factor for x in w], 1.0
    if case["scaling"] == "base":
        # a larger base that leaves the first pair's frequency and divides the last one's by the factor
        base = theta * factor ** (rot / max(rot - 2.0, 1.0))
        return [base ** (-2.0 * i / rot) for i in range(half)], 1.0
    if case["scaling"] == "bands":
        # wavelengths up to old / 4 stay, from old on they grow by the factor, between them a blend
        out = []
        for x in w:
            turns = old * x / (2.0 * math.pi)
            keep = min(1.0, max(0.0, (turns - 1.0) / (4.0 - 1.0)))
            out.append(x * keep + x / factor * (1.0 - keep))
        return out, 1.0
    if case["scaling"] == "ramp":
        # the blend is linear in the pair's index, between the pairs that turn 32 times and once over the old length
        def pair(turns):
            return rot * math.log(old / (turns * 2.0 * math.pi)) / (2.0 * math.log(theta))
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), half - 1)
        hi = hi + 0.001 if hi == lo else hi
        out = []
        for i, x in enumerate(w):
            slow = min(1.0, max(0.0, (i - lo) / (hi - lo)))
            out.append(x * (1.0 - slow) + x / factor * slow)
        return out, 0.1 * math.log(factor) + 1.0
    return w, 1.0


def _rows(gen, n, H, hd, spread):
    """n rows of H heads: channels of unequal size, a few of them large, as keys have them."""
    size = torch.exp(spread * torch.randn(H, hd, generator=gen, device="cuda"))
    drift = torch.randn(1 + n // PAGE, H, hd, generator=gen, device="cuda").repeat_interleave(PAGE, dim=0)[:n]
    return torch.randn(n, H, hd, generator=gen, device="cuda").add_(drift, alpha=0.7).mul_(size)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case}
    if case["op"] == "pages":
        held, keep, new = _requests(case, seed)
        for name, v in (("held", held), ("keep", keep), ("new", new)):
            st[name] = torch.tensor(v, dtype=torch.int32, device="cuda")
        used = [_pages(h) for h in held]
        grow = sum(max(0, _pages(k + n) - u) for k, n, u in zip(keep, new, used))
        n_pages = sum(used) + grow + 7
        order = torch.randperm(n_pages, generator=gen, device="cuda").int()
        table = torch.zeros(case["n_req"], case["width"], dtype=torch.int32, device="cuda")
        mask = torch.arange(case["width"], device="cuda") < torch.tensor(used, device="cuda")[:, None]
        table[mask] = order[:sum(used)]
        st["table"], st["free"] = table, torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        st["free"][:n_pages - sum(used)] = order[sum(used):]
        st["n_free"] = torch.tensor([n_pages - sum(used)], dtype=torch.int32, device="cuda")
        st["n_tok"] = sum(new)
    elif case["op"] == "rope":
        n, dt = case["n_tok"], torch.float32 if case["dtype"] == "f32" else torch.float16
        st["q"] = (1.5 * torch.randn(n, case["n_qh"], case["hd"], generator=gen, device="cuda")).to(dt)
        st["k"] = (1.5 * torch.randn(n, case["n_kvh"], case["hd"], generator=gen, device="cuda")).to(dt)
        st["positions"] = torch.randint(0, case["far"], (n,), generator=gen, device="cuda", dtype=torch.int32)
        freq, st["mag"] = _frequencies(case)
        st["freq"] = torch.tensor(freq, dtype=torch.float64, device="cuda")
    elif case["op"] == "write":
        n, H, hd = case["n_tok"], case["n_kvh"], case["hd"]
        dt = torch.float32 if case["src"] == "f32" else torch.float16
        st["k_src"], st["v_src"] = _rows(gen, n, H, hd, 0.5).to(dt), _rows(gen, n, H, hd, 0.2).to(dt)
        if case["kind"] == "decode":   # each token in a page of its own request
            st["n_pages"] = n + 3
            page = torch.randperm(n + 3, generator=gen, device="cuda")[:n]
            st["slots"] = page * PAGE + torch.randint(0, PAGE, (n,), generator=gen, device="cuda")
        else:                          # consecutive positions from the middle of a page on
            st["n_pages"] = _pages(n + 33) + 3
            page = torch.randperm(st["n_pages"], generator=gen, device="cuda")
            i = torch.arange(33, 33 + n, device="cuda")
            st["slots"] = page[i // PAGE] * PAGE + i % PAGE
    else:
        held, rows = _lengths(case, seed)
        H, hd, R = case["n_kvh"], case["hd"], case["n_req"]
        used = [_pages(h) for h in held]
        st["n_pages"] = sum(used) + 3
        order = torch.randperm(st["n_pages"], generator=gen, device="cuda").int()
        st["table"] = torch.zeros(R, max(used), dtype=torch.int32, device="cuda")
        mask = torch.arange(max(used), device="cuda") < torch.tensor(used, device="cuda")[:, None]
        st["table"][mask] = order[:sum(used)]
        st["held"] = torch.tensor(held, dtype=torch.int32, device="cuda")
        st["q_start"] = torch.tensor([0] + rows, dtype=torch.int32, device="cuda").cumsum(0).int()
        st["slots"] = torch.cat([st["table"][r, torch.arange(h, device="cuda") // PAGE].long() * PAGE
                                 + torch.arange(h, device="cuda") % PAGE for r, h in enumerate(held) if h])
        st["q"] = torch.randn(sum(rows), case["n_qh"], hd, generator=gen, device="cuda") * 1.5
        st["k_src"], st["v_src"] = _rows(gen, sum(held), H, hd, 0.5), _rows(gen, sum(held), H, hd, 0.2)
    return st


def _fill(st, with_rows):
    """The plain form's cache of an attention case: packed codes and scales by slot, a head at a time."""
    c = st["case"]
    H, hd = c["n_kvh"], c["hd"]
    for w in "kv":
        st[w] = torch.zeros(st["n_pages"] * PAGE, H, hd // 2, dtype=torch.uint8, device="cuda")
        st[w + "scale"] = torch.zeros(st["n_pages"] * PAGE, H, hd // GROUP, dtype=torch.float16, device="cuda")
        if with_rows:
            for h in range(H):
                code, scale = _quantise(st[w + "_src"][:, h], c["fmt"])
                st[w][st["slots"], h], st[w + "scale"][st["slots"], h] = _pack(code), scale
            del st[w + "_src"]


def prepare(case, seed):
    st = _inputs(case, seed)
    op = case["op"]
    if not own:
        if op in ("write", "attend"):
            _fill(st, op == "attend")
        return st
    from block_quantized_gemv_nt_gb300 import engine, nt
    st["ctx"] = nt.Context(torch.cuda.current_device())
    if op == "pages":
        st["pages"] = engine.KV4Pages(st["ctx"], case["n_req"], case["width"], st["free"].numel(),
                                      buffers={n: st[n] for n in ("table", "held", "free", "n_free")})
        st["held_out"], st["n_free_out"] = torch.empty_like(st["held"]), torch.empty_like(st["n_free"])
        st["q_start"] = torch.empty(case["n_req"] + 1, dtype=torch.int32, device="cuda")
        st["slots"] = torch.empty(st["n_tok"], dtype=torch.int64, device="cuda")
        st["positions"] = torch.empty(st["n_tok"], dtype=torch.int32, device="cuda")
    elif op == "rope":
        kind = {"none": nt.ROPE_PLAIN, "linear": nt.ROPE_LINEAR, "base": nt.ROPE_BASE, "bands": nt.ROPE_BANDS,
                "ramp": nt.ROPE_RAMP}[case["scaling"]]
        st["rope"] = engine.Rope(st["ctx"], case["hd"], case["rot"],
                                 nt.ROPE_PAIRS if case["layout"] == "pairs" else nt.ROPE_HALVES, theta=500000.0,
                                 scaling=kind, factor=8.0, old_len=8192)
        st["q_out"], st["k_out"] = torch.empty_like(st["q"]), torch.empty_like(st["k"])
    else:
        fmt = nt.KV4_I4 if case["fmt"] == "i4" else nt.KV4_E2M1
        st["cache"] = engine.KV4Cache(st["ctx"], fmt, case["n_kvh"], case["hd"], st["n_pages"])
        if op == "write":
            st["k_out"], st["v_out"] = torch.empty_like(st["k_src"]), torch.empty_like(st["v_src"])
        else:
            st["cache"].append(st.pop("k_src"), st.pop("v_src"), st["slots"])
            st["out"] = torch.empty_like(st["q"])
    return st


def run(st):
    op = st["case"]["op"]
    if not own:
        return {"pages": _plain_pages, "rope": _plain_rope, "write": _plain_write, "attend": _plain_attend}[op](st)
    if op == "pages":
        st["pages"].step(st["new"], st["q_start"], st["slots"], st["positions"], keep=st["keep"],
                         held_out=st["held_out"], n_free_out=st["n_free_out"])
        return {"table": st["table"], "free": st["free"], "n_free": st["n_free_out"], "held": st["held_out"],
                "q_start": st["q_start"], "slots": st["slots"], "positions": st["positions"]}
    if op == "rope":
        st["rope"].rotate((st["q"], st["q_out"]), (st["k"], st["k_out"]), positions=st["positions"])
        return [st["q_out"], st["k_out"]]
    if op == "write":
        st["cache"].append(st["k_src"], st["v_src"], st["slots"])
        st["cache"].read(st["k_out"], st["v_out"], st["slots"])
        return [st["k_out"], st["v_out"]]
    st["cache"].attend(st["q"], st["out"], st["q_start"], st["held"], st["table"])
    return st["out"]


# ---- the definition in 64 bits --------------------------------------------------------
def _exact_pages(st):
    table, free = st["table"].cpu().tolist(), st["free"].cpu().tolist()
    top = int(st["n_free"])
    held, keep, new = (st[n].cpu().tolist() for n in ("held", "keep", "new"))
    for r, h in enumerate(held):
        for j in range(_pages(keep[r] + new[r]), _pages(h)):
            free[top] = table[r][j]
            top += 1
    left, asked, q_start, slots, positions, out = top, 0, [0], [], [], []
    for r, h in enumerate(held):
        have, want = _pages(h), _pages(keep[r] + new[r])
        asked += max(0, want - have)
        ok = want <= have or asked <= top
        if ok and want > have:
            table[r][have:want] = free[left - (want - have):left][::-1]
            left -= want - have
        out.append(keep[r] + new[r] if ok else h)
        for p in range(keep[r], keep[r] + new[r]):
            slots.append(table[r][p // PAGE] * PAGE + p % PAGE if ok else -1)
            positions.append(p)
        q_start.append(len(slots))
    i32 = {"dtype": torch.int32, "device": "cuda"}
    return {"table": torch.tensor(table, **i32), "free": torch.tensor(free, **i32), "n_free": torch.tensor([left], **i32),
            "held": torch.tensor(out, **i32), "q_start": torch.tensor(q_start, **i32),
            "slots": torch.tensor(slots, dtype=torch.int64, device="cuda"), "positions": torch.tensor(positions, **i32)}


def _exact_rope(st):
    c, half = st["case"], st["case"]["rot"] // 2
    turn = torch.polar(torch.full((c["n_tok"], half), st["mag"], dtype=torch.float64, device="cuda"),
                       st["positions"].double()[:, None] * st["freq"])[:, None]
    outs = []
    for w in ("q", "k"):
        y = st[w].double()
        lo, hi = ((slice(0, c["rot"], 2), slice(1, c["rot"], 2)) if c["layout"] == "pairs"
                  else (slice(0, half), slice(half, c["rot"])))
        z = torch.complex(y[..., lo], y[..., hi]) * turn
        y[..., lo], y[..., hi] = z.real, z.imag
        outs.append(y)
    return outs


def _exact_round(x, digits, least):
    """x at the nearest number of `digits` significant bits, then at the nearest multiple of `least`, ties to even."""
    drop = 53 - digits
    bits = x.view(torch.int64)
    bits = (bits + (1 << (drop - 1)) - 1 + ((bits >> drop) & 1)) >> drop << drop
    return torch.round(bits.view(torch.float64) / least) * least


def _exact_grid(x, fmt):
    """The values over the scale, and the scale: x [..., groups, 32] in 64 bits."""
    if fmt == "i4":
        top = x.abs().amax(dim=-1, keepdim=True)
        d = torch.where((x == top).any(dim=-1, keepdim=True), -top, top) / 8
    else:
        d = x.abs().amax(dim=-1, keepdim=True) / 6
    d = _exact_round(d.clamp(-TOP_SCALE, TOP_SCALE), 8, 2.0 ** -24)
    y = torch.where(d == 0, torch.zeros_like(x), x / d)
    if fmt == "i4":
        return torch.round(y).clamp(-8, 7), d
    mag = y.abs().clamp(max=6.0)
    step = torch.where(mag < 2, 0.5, torch.where(mag < 4, 1.0, 2.0)).double()
    return torch.copysign(torch.round(mag / step) * step, y), d


def _exact_values(x, fmt):
    v, d = _exact_grid(x.double().unflatten(-1, (-1, GROUP)), fmt)
    return (v * d).flatten(-2)


def _exact_attend(st):
    c = st["case"]
    H, G, hd = c["n_kvh"], c["n_qh"] // c["n_kvh"], c["hd"]
    held, rows = st["held"].tolist(), (st["q_start"][1:] - st["q_start"][:-1]).tolist()
    q = st["q"].double().view(-1, H, G, hd)
    out = torch.zeros_like(q)
    at, row = 0, 0
    for n, nq in zip(held, rows):
        for h in range(H if nq else 0):
            k, v = (_exact_values(st[w + "_src"][at:at + n, h], c["fmt"]) for w in "kv")
            for i in range(nq):
                m = n - (nq - 1 - i)
                if m > 0:
                    s = q[row + i, h] @ k[:m].T / math.sqrt(hd)
                    out[row + i, h] = torch.softmax(s, dim=-1) @ v[:m]
        at, row = at + n, row + nq
    return out.view(-1, H * G, hd)


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "write":
        return [_exact_values(st[w + "_src"], case["fmt"]) for w in "kv"]
    return {"pages": _exact_pages, "rope": _exact_rope, "attend": _exact_attend}[case["op"]](st)
