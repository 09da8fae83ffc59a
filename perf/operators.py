"""Cases of the operators around the paged cache: attention over a cache held
in four bits, page management, and rotary positions with several axes.

A case names an operator ("op") and a way of calling it ("mode") with sizes.
``run`` computes it in plain torch operations, or with ``own`` through the
framework's calls.  ``exact`` gives the values of the definitions in 64 bits.

Four-bit entries: element = e2m1(code) * e4m3(block scale) * tensor scale, one
block scale per 16 elements.  Stored for x: y = fp32(x * fp32(1 / scale)),
block scale = e4m3(fp32(max |y| / 6)), code = e2m1(fp32(y / block scale)),
rounded to nearest even and clamped.  Element 2j sits in the low half of byte
j.  Codes are [slots, Hkv, D/2], block scales [Hkv, slots, D/16].
"""
import math

import torch

own = False

EPS = 1e-6
THETA = 1e6
K_SCALE = 0.03125
V_SCALE = 0.0625
DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
E2M1_MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


# ------------------------------------------------------------------ cases
def _c4(name, mode, batch, new, lo, hi, hq, hkv, d, page):
    return {"name": name, "op": "cache4", "mode": mode, "batch": batch, "new": new, "lo": lo, "hi": hi, "hq": hq,
            "hkv": hkv, "d": d, "page": page}


def _pg(name, mode, pages, page, hkv, d, kind, rows, ways, lo, hi):
    return {"name": name, "op": "pages", "mode": mode, "pages": pages, "page": page, "hkv": hkv, "d": d, "type": kind,
            "rows": rows, "ways": ways, "lo": lo, "hi": hi}


def _ax(name, mode, tokens, lo, hi, hq, hkv, d, sections, inter):
    return {"name": name, "op": "axes", "mode": mode, "tokens": tokens, "lo": lo, "hi": hi, "hq": hq, "hkv": hkv,
            "d": d, "sections": sections, "interleaved": inter}


def listed():
    return [
        # one user's next token over a short chat: the latency of a call
        _c4("decode4 one short", "decode", 1, 1, 777, 777, 32, 8, 128, 64),
        # the framework's decode batch: 64 requests, cached lengths 512 .. 8192
        _c4("decode4 batch", "decode", 64, 1, 512, 8192, 32, 8, 128, 64),
        # long documents: few requests, each split over the whole card
        _c4("decode4 long", "decode", 16, 1, 30001, 65000, 64, 8, 128, 128),
        # small heads, odd lengths, contiguous regions
        _c4("decode4 small heads", "decode", 37, 1, 3, 2500, 16, 2, 64, 0),
        # chunks of prompts over their cached prefixes (ragged)
        _c4("prefill4 chunks", "prefill", 4, 300, 100, 6000, 32, 4, 128, 64),
        # a prompt sampled eight ways: its pages shared, the open page copied
        _pg("fork one prompt", "fork", 512, 64, 8, 128, "bf16", 1, 8, 1000, 1000),
        # a batch of prompts, each sampled several ways, over a one-byte cache
        _pg("fork batch", "fork", 6000, 64, 8, 128, "e4m3", 96, 4, 333, 5000),
        # requests finish and others take their pages: the host loop's call
        _pg("free and reserve", "turnover", 20000, 64, 1, 64, "bf16", 256, 0, 100, 4000),
        # a fragmented pool of four-bit pages packed to the front
        _pg("compact four-bit", "compact", 6000, 64, 8, 128, "e2m1", 120, 0, 700, 2900),
        # pages copied within a bf16 pool
        _pg("copy pages", "copy", 3000, 64, 8, 128, "bf16", 1400, 0, 0, 0),
        # a long prompt with images: text runs and patch grids
        _ax("axes long prompt", "prepare", 32768, 0, 0, 32, 8, 128, "24,20,20", True),
        # a batch's next tokens after multimodal prompts
        _ax("axes decode", "decode", 64, 100, 2000, 32, 8, 128, "16,24,24", False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("cache4", "cache4", "pages", "pages", "axes"))
    heads = rng.choice(((32, 8, 128), (16, 2, 64), (8, 8, 128), (64, 8, 128), (8, 4, 64), (6, 3, 128), (4, 1, 128)))
    if op == "cache4":
        page = rng.choice((0, 64, 64, 128, 256))
        if rng.random() < 0.3:
            hi = _log(rng, 20, 5000)
            c = _c4("", "prefill", rng.randint(1, 4), _log(rng, 2, 300), rng.randint(0, hi), hi, *heads, page)
            c["hkv"] = max(c["hq"] // 8, min(c["hkv"], 4)) if c["hq"] % 4 == 0 else c["hkv"]
        else:
            batch = _log(rng, 1, 100)
            hi = _log(rng, 10, min(60000, 400000 // batch))
            c = _c4("", "decode", batch, 1, rng.randint(0, hi), hi, *heads, page)
    elif op == "pages":
        mode = rng.choice(("copy", "fork", "turnover", "compact"))
        kind, page = rng.choice(("bf16", "e4m3", "e2m1")), rng.choice((64, 64, 128))
        rows = _log(rng, 1, 100)
        hi = _log(rng, 10, 3000)
        c = _pg("", mode, 0, page, heads[1], heads[2], kind, rows, rng.randint(1, 4) if mode == "fork" else 0,
                rng.randint(1, hi), hi)
        if mode == "copy":
            c["rows"] = _log(rng, 1, 600)
            c["lo"] = c["hi"] = 0
            c["pages"] = 2 * c["rows"] + rng.randint(1, 200)
        else:
            c["pages"] = rows * (hi // page + 2 + c["ways"]) * 3 // 2 + rng.randint(3, 99)
    else:
        d = heads[2]
        a = rng.randint(d // 8, d // 6)
        b = rng.randint(d // 8, d // 6)
        sec = "%d,%d,%d" % (d // 2 - a - b, a, b)
        if rng.random() < 0.5:
            c = _ax("", "prepare", _log(rng, 1, 18000), 0, 0, *heads, sec, rng.random() < 0.5)
        else:
            hi = _log(rng, 10, 2000)
            c = _ax("", "decode", _log(rng, 1, 64), rng.randint(0, hi), hi, *heads, sec, rng.random() < 0.5)
    del c["name"]
    return c


def _spread(lo, hi, n):
    """n whole numbers over [lo, hi], evenly spaced and in a mixed order."""
    if n == 1:
        return [hi]
    step = next(s for s in (7, 11, 13, 17, 19, 23) if n % s)
    return [lo + (hi - lo) * ((i * step) % n) // (n - 1) for i in range(n)]


def _lens(case):
    """(cached lengths, new lengths) of a case's requests."""
    B = case["batch"]
    cached = _spread(case["lo"], case["hi"], B)
    new = [1] * B if case["mode"] == "decode" else _spread(max(1, case["new"] // 3), case["new"], B)
    return cached, new


def _row_bytes(kind, d):
    """Bytes of one head's entry: codes, block scales."""
    return {"bf16": (2 * d, 0), "e4m3": (d, 0), "e2m1": (d // 2, d // 16)}[kind]


def work(case):
    d = case["d"]
    hkv = case["hkv"]
    if case["op"] == "cache4":
        cached, new = _lens(case)
        hq = case["hq"]
        n, pairs = sum(new), sum(m * c + m * (m + 1) // 2 for c, m in zip(cached, new))
        entry = 2 * hkv * sum(_row_bytes("e2m1", d))
        # cache read, qkv read, out written, new entries written and given back
        return {"bytes": sum(cached) * entry + n * ((hq + 2 * hkv) * d * 2 + hq * d * 2 + entry + 2 * hkv * d * 2),
                "flops": 4.0 * pairs * hq * d}
    if case["op"] == "pages":
        per_slot = 2 * hkv * sum(_row_bytes(case["type"], d))
        s = _pool_plan(case)
        ints = 2 * 4 * (s["rows"] * s["ppr"] + case["pages"] + s["rows"])
        if case["mode"] == "copy":
            return {"bytes": 2 * case["rows"] * case["page"] * per_slot + 8 * case["rows"], "flops": 0}
        if case["mode"] == "fork":
            tails = sum(c % case["page"] for c in s["lens"]) * case["ways"]
            return {"bytes": 2 * tails * per_slot + ints, "flops": 0}
        if case["mode"] == "compact":
            # in the mean: the share of live pages that lie behind the live count
            live = s["live"]
            moved = live * (1 - live / case["pages"])
            return {"bytes": 2 * moved * case["page"] * per_slot + ints, "flops": 0}
        return {"bytes": ints, "flops": 0}
    n, hq = case["tokens"], case["hq"]
    if case["mode"] == "prepare":
        return {"bytes": n * ((hq + 2 * hkv) * d * 2 * 2 + 12), "flops": 6.0 * n * (hq + hkv) * d}
    cached = _spread(case["lo"], case["hi"], n)
    return {"bytes": sum(cached) * hkv * d * 4 + n * ((hq + 2 * hkv) * d * 2 + 2 * hkv * d * 2 + hq * d * 2 + 12),
            "flops": 4.0 * sum(c + 1 for c in cached) * hq * d}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _norm_weights(g, d):
    return (1 + 0.1 * _randn(g, d)).bfloat16()


def _quantise(x, scale):
    """(codes, block scales) of x [..., D] fp32: uint8 [..., D/2], uint8 [..., D/16]."""
    y = (x * (1.0 / scale)).view(*x.shape[:-1], -1, 16)
    # divisors on the device: a number as divisor is turned into a product with its reciprocal
    s = (y.abs().amax(-1) / torch.full((1,), 6.0, device=DEV)).clamp_(max=448.0).to(torch.float8_e4m3fn)
    sf = s.float()[..., None]
    z = torch.where(sf > 0, y / sf, torch.zeros_like(y))
    m = z.abs()
    idx = torch.zeros_like(m, dtype=torch.uint8)
    for i, mid in enumerate(E2M1_MIDS):  # a tie goes to the code with an even mantissa bit
        idx += (m >= mid) if i % 2 else (m > mid)
    code = (idx + 8 * torch.signbit(z).to(torch.uint8)).view(*x.shape[:-1], -1, 2)
    return code[..., 0] + 16 * code[..., 1], s.view(torch.uint8)


def _values(codes, scales, scale):
    """fp32 entries of codes [..., D/2] with block scales [..., D/16]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1)
    v = v.view(*codes.shape[:-1], -1, 16) * scales.view(torch.float8_e4m3fn).float()[..., None]
    return v.view(*codes.shape[:-1], -1) * scale


def _tables(g, lens, page, spare):
    """A page table of pages drawn at random, and the pool's page count."""
    need = [-(-c // page) for c in lens]
    total = sum(need) + spare
    perm = torch.randperm(total, generator=g, device=DEV).int()
    ppr = max(need)
    at = torch.tensor([sum(need[:b]) for b in range(len(need))], device=DEV)[:, None] + torch.arange(ppr, device=DEV)
    live = torch.arange(ppr, device=DEV) < torch.tensor(need, device=DEV)[:, None]
    return torch.where(live, perm[at.clamp(max=total - 1)], torch.full_like(perm[:1], -1)).contiguous(), total


def _prepare_cache4(case, g):
    d, hq, hkv, page = case["d"], case["hq"], case["hkv"], case["page"]
    cached, new = _lens(case)
    B, N = len(cached), sum(new)
    full = [c + n for c, n in zip(cached, new)]
    st = {"case": case, "max_new": max(new), "max_cached": max(cached), "max_len": max(full)}
    if page:
        st["table"], pages = _tables(g, full, page, 5)
        slots = pages * page
        st["base"] = torch.zeros(B, dtype=torch.int64, device=DEV)
        st["cap"] = torch.full((B,), st["table"].shape[1] * page, dtype=torch.int32, device=DEV)
    else:
        st["table"] = None
        starts = [3 + sum(full[:b]) + 3 * b for b in range(B)]
        slots = starts[-1] + full[-1] + 3
        st["base"] = torch.tensor(starts, dtype=torch.int64, device=DEV)
        st["cap"] = torch.tensor(full, dtype=torch.int32, device=DEV)
    for n, scale in (("k", K_SCALE), ("v", V_SCALE)):
        codes, s = _quantise(_randn(g, slots, hkv, d), scale)
        st[n] = codes.contiguous()
        st[n + "s"] = s.transpose(0, 1).contiguous()
        del codes, s
    st["qkv"] = _randn(g, N, (hq + 2 * hkv) * d).bfloat16()
    st["qw"], st["kw"] = _norm_weights(g, d), _norm_weights(g, d)
    st["lens"] = torch.tensor(cached, dtype=torch.int32, device=DEV)
    st["cu"] = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32, device=DEV)
    # the packed tokens' requests and positions, which a scheduler has at hand
    st["req"] = torch.tensor([b for b in range(B) for _ in range(new[b])], device=DEV)
    st["pos"] = torch.tensor([cached[b] + j for b in range(B) for j in range(new[b])], device=DEV)
    return st


def _pool_plan(case):
    """Sizes of a page case that do not depend on the seed."""
    page, rows = case["page"], case["rows"]
    if case["mode"] == "copy":
        return {"rows": 1, "ppr": 1, "lens": [], "need": [], "live": 0}
    lens = _spread(case["lo"], case["hi"], rows)
    need = [-(-c // page) for c in lens]
    # room for the rows that fork or start anew
    total = rows * (1 + case["ways"])
    return {"rows": total, "ppr": max(need) + 2, "lens": lens, "need": need, "live": sum(need)}


def _prepare_pages(case, g):
    P, page, hkv, d, kind = case["pages"], case["page"], case["hkv"], case["d"], case["type"]
    st = {"case": case}
    shape = (P * page, hkv)
    for n in ("k", "v"):
        if kind == "bf16":
            st[n] = _randn(g, *shape, d).bfloat16()
        else:  # codes: all finite values
            w = d if kind == "e4m3" else d // 2
            st[n] = torch.randint(0, 126 if kind == "e4m3" else 256, (*shape, w), generator=g, device=DEV, dtype=torch.uint8)
        if kind == "e2m1":
            st[n + "s"] = torch.randint(0, 126, (hkv, P * page, d // 16), generator=g, device=DEV, dtype=torch.uint8)
    perm = torch.randperm(P, generator=g, device=DEV).int()
    plan = _pool_plan(case)
    if case["mode"] == "copy":
        n = case["rows"]
        st["src"], st["dst"] = perm[:n].contiguous(), perm[n:2 * n].contiguous()
        st["start"] = torch.zeros(P + 2, dtype=torch.int32, device=DEV)
        st["now"] = st["start"].clone()
        return st
    rows, ppr, lens, need = plan["rows"], plan["ppr"], plan["lens"], plan["need"]
    # table [rows, ppr], ref_count [P] and cache_lens [rows] in one buffer that a pass starts from
    start = torch.full((rows * ppr + P + rows,), -1, dtype=torch.int32, device=DEV)
    table, ref, ln = start[:rows * ppr].view(rows, ppr), start[rows * ppr:rows * ppr + P], start[rows * ppr + P:]
    at = torch.tensor([sum(need[:b]) for b in range(len(need))], device=DEV)[:, None] + torch.arange(ppr, device=DEV)
    live = torch.arange(ppr, device=DEV) < torch.tensor(need, device=DEV)[:, None]
    table[:len(lens)] = torch.where(live, perm[at.clamp(max=P - 1)], table[:len(lens)])
    ref.zero_()
    ref[perm[:plan["live"]].long()] = 1
    ln.zero_()
    ln[:len(lens)] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    if case["mode"] == "compact" and len(lens) > 1:  # some rows share their first page, as forks leave them
        half = len(lens) // 2
        ref[table[half:2 * half, 0].long()] -= 1
        table[half:2 * half, 0] = table[:half, 0]
        ref[table[:half, 0].long()] += 1
    st["start"], st["now"] = start, start.clone()
    now = st["now"]
    st["table"], st["ref"], st["lens"] = (now[:rows * ppr].view(rows, ppr), now[rows * ppr:rows * ppr + P],
                                          now[rows * ppr + P:])
    n = len(lens)
    if case["mode"] == "fork":
        st["src"] = torch.arange(n, dtype=torch.int32, device=DEV).repeat_interleave(case["ways"])
        st["dst"] = torch.arange(n, rows, dtype=torch.int32, device=DEV)
    if case["mode"] == "turnover":  # every third request ends; the others and the new ones get room
        st["ended"] = torch.arange(0, n, 3, dtype=torch.int32, device=DEV)
        st["grow"] = torch.randperm(n, generator=g, device=DEV).int()
        st["more"] = torch.randint(1, case["page"] + 1, (n,), generator=g, device=DEV, dtype=torch.int32)
    return st


def _positions(n, g):
    """int32 [3, n]: runs of 100 text tokens, each followed by a 16 x 24 grid of patches."""
    i = torch.arange(n, device=DEV)
    base0 = torch.randint(0, 5000, (1,), generator=g, device=DEV)
    text, rows, cols = 100, 16, 24
    turn, off = i // (text + rows * cols), i % (text + rows * cols)
    base = base0 + turn * (text + cols)
    patch = off - text
    t = torch.where(off < text, base + off, base + text)
    h = torch.where(off < text, base + off, base + text + patch // cols)
    w = torch.where(off < text, base + off, base + text + patch % cols)
    return torch.stack((t, h, w)).int()


def _prepare_axes(case, g):
    n, d, hq, hkv = case["tokens"], case["d"], case["hq"], case["hkv"]
    st = {"case": case, "qkv": _randn(g, n, (hq + 2 * hkv) * d).bfloat16(), "qw": _norm_weights(g, d),
          "kw": _norm_weights(g, d), "positions": _positions(n, g)}
    if case["mode"] == "prepare":
        cached, slots = [0], n
        st["cu"] = torch.tensor([0, n], dtype=torch.int32, device=DEV)
        st["base"] = torch.zeros(1, dtype=torch.int64, device=DEV)
        st["cap"] = torch.tensor([n], dtype=torch.int32, device=DEV)
        st["slots"] = torch.arange(n, device=DEV)
        st["q"] = torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV)
    else:
        cached = _spread(case["lo"], case["hi"], n)
        starts = [sum(cached[:b]) + b for b in range(n)]
        slots = starts[-1] + cached[-1] + 1
        st["base"] = torch.tensor(starts, dtype=torch.int64, device=DEV)
        st["cap"] = torch.tensor([c + 1 for c in cached], dtype=torch.int32, device=DEV)
        st["slots"] = st["base"] + torch.tensor(cached, device=DEV)
        st["max_cached"] = max(cached)
    st["lens"] = torch.tensor(cached, dtype=torch.int32, device=DEV)
    st["k"], st["v"] = _randn(g, slots, hkv, d).bfloat16(), _randn(g, slots, hkv, d).bfloat16()
    return st


def prepare(case, seed):
    return {"cache4": _prepare_cache4, "pages": _prepare_pages, "axes": _prepare_axes}[case["op"]](case, _gen(seed))


# ------------------------------------------------------------------ plain forms
def _rotated(x, w, angles):
    """RMSNorm and rotate-half of x [N, H, D] fp32 at angles [N, D/2] (64 bits)."""
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    c, s = angles.cos().float()[:, None], angles.sin().float()[:, None]
    a, b = x.chunk(2, -1)
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def _freqs(d):
    return torch.pow(torch.tensor(THETA, dtype=torch.float64, device=DEV),
                     -2.0 * torch.arange(d // 2, dtype=torch.float64, device=DEV) / d)


def _split(st, hq, hkv, d):
    x = st["qkv"].float().view(-1, hq + 2 * hkv, d)
    return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]


def _attend(q, keys, vals, see):
    """softmax(q k^T / sqrt(D)) v: q [B, n, Hq, D], keys and vals [B, L, Hkv, D], see [B, n, L]."""
    B, n, hq, d = q.shape
    hkv = keys.shape[2]
    q = q.view(B, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, d)
    s = torch.matmul(q, keys.permute(0, 2, 3, 1)).view(B, hkv, -1, n, keys.shape[1]) * (1.0 / math.sqrt(d))
    s = s.masked_fill(~see[:, None, None], float("-inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, hkv, -1, keys.shape[1]), vals.permute(0, 2, 1, 3))
    return o.view(B, hkv, hq // hkv, n, d).permute(0, 3, 1, 2, 4).reshape(B, n, hq * d)


def _plain_cache4(st):
    c = st["case"]
    d, hq, hkv, page = c["d"], c["hq"], c["hkv"], c["page"]
    q, k, v = _split(st, hq, hkv, d)
    angles = st["pos"].double()[:, None] * _freqs(d)
    q, k = _rotated(q, st["qw"], angles), _rotated(k, st["kw"], angles)
    B, L, n = st["lens"].numel(), st["max_len"], st["max_new"]
    pos = torch.arange(L, device=DEV)
    if page:
        slots = st["table"].long()[:, pos // page].clamp(min=0) * page + pos % page
    else:
        slots = (st["base"][:, None] + pos).clamp(max=st["k"].shape[0] - 1)
    at = slots[st["req"], st["pos"]]
    new = []
    for name, x, scale in (("k", k, K_SCALE), ("v", v, V_SCALE)):
        codes, s = _quantise(x, scale)
        st[name][at] = codes
        st[name + "s"][:, at] = s.transpose(0, 1)
        new.append(_values(codes, s, scale).bfloat16())
    cu, lens = st["cu"].long(), st["lens"].long()
    at_q = (cu[:-1, None] + torch.arange(n, device=DEV)).clamp(max=q.shape[0] - 1)
    see = pos[None, None, :] <= (lens[:, None] + torch.arange(n, device=DEV))[:, :, None]
    keys = _values(st["k"][slots], st["ks"][:, slots].permute(1, 2, 0, 3), K_SCALE)
    vals = _values(st["v"][slots], st["vs"][:, slots].permute(1, 2, 0, 3), V_SCALE)
    # slots past a request's end belong to others: no part in its sums
    ends = (lens + cu[1:] - cu[:-1])[:, None, None, None]
    vals = vals.masked_fill(pos[None, :, None, None] >= ends, 0.0)
    keys = keys.masked_fill(pos[None, :, None, None] >= ends, 0.0)
    o = _attend(q[at_q], keys, vals, see)
    out = o[st["req"], st["pos"] - lens[st["req"]]].bfloat16()
    return {"out": out, "k_new": new[0], "v_new": new[1]}


def _pools(st):
    P, page = st["case"]["pages"], st["case"]["page"]
    t = [st[n].view(P, page, *st[n].shape[1:]) for n in ("k", "v")]
    t += [st[n].view(-1, P, page, st[n].shape[2]).permute(1, 2, 0, 3) for n in ("ks", "vs") if n in st]
    return t


def _returned(st):
    r = {n: st[n] for n in ("k", "v", "ks", "vs") if n in st}
    if st["case"]["mode"] == "turnover":  # no entry moves
        r = {}
    if "table" in st:
        r |= {"table": st["table"], "ref": st["ref"], "lens": st["lens"]}
    return r


def _lowest_free(ref, n):
    return torch.argsort((ref > 0).int(), stable=True)[:n]


def _plain_pages(st):
    c = st["case"]
    page = c["page"]
    st["now"].copy_(st["start"])
    if c["mode"] == "copy":
        for t in _pools(st):
            t[st["dst"].long()] = t[st["src"].long()]
        return _returned(st)
    table, ref, lens = st["table"], st["ref"], st["lens"]
    ppr = table.shape[1]
    j = torch.arange(ppr, device=DEV)
    one = torch.ones(1, dtype=torch.int32, device=DEV)
    if c["mode"] == "fork":
        src, dst = st["src"].long(), st["dst"].long()
        ln = lens[src].long()
        whole, rest = ln // page, ln % page
        need = rest > 0
        # the n-th request with an open page gets the n-th free page; the others are
        # given pages behind those, so that no two write to the same one (nothing changes there)
        rank = torch.where(need, torch.cumsum(need, 0), need.sum() + torch.cumsum(~need, 0)) - 1
        fresh = _lowest_free(ref, src.numel())[rank]
        rows = table[src]
        shared = j < whole[:, None]
        tail = rows.gather(1, whole[:, None])[:, 0].long()
        rows = torch.where(shared, rows, torch.full_like(rows, -1))
        rows = torch.where((j == whole[:, None]) & need[:, None], fresh[:, None].int(), rows)
        ref.index_add_(0, torch.where(shared, rows, 0).long().view(-1), shared.view(-1).int())
        ref.index_add_(0, fresh, need.int())
        table[dst] = rows
        lens[dst] = ln.int()
        used = torch.arange(page, device=DEV) < rest[:, None]
        for t in _pools(st):
            keep = used.view(*used.shape, *([1] * (t.dim() - 2)))
            t[fresh] = torch.where(keep, t[tail.clamp(min=0)], t[fresh])
    elif c["mode"] == "turnover":
        ended = st["ended"].long()
        old = table[ended].view(-1)
        ref.index_add_(0, old.clamp(min=0).long(), -(old >= 0).int())
        table[ended] = -1
        lens[ended] = 0
        rows = st["grow"].long()
        have, want = -(-lens[rows] // page), -(-(lens[rows] + st["more"]) // page)
        t = table[rows]
        wanted = (j >= have[:, None]) & (j < want[:, None]) & (t < 0)
        rank = torch.cumsum(wanted.view(-1), 0) - 1
        most = rows.numel() * 2
        fresh = _lowest_free(ref, most)[rank.clamp(min=0, max=most - 1)].view(t.shape).int()
        table[rows] = torch.where(wanted, fresh, t)
        ref.index_add_(0, torch.where(wanted, fresh, 0).long().view(-1), wanted.view(-1).int())
    else:
        live = ref > 0
        n_live = live.sum()
        p = torch.arange(ref.numel(), device=DEV)
        moved, holes = (live & (p >= n_live)).nonzero()[:, 0], (~live & (p < n_live)).nonzero()[:, 0]
        for t in _pools(st):
            t[holes] = t[moved]
        to = p.int()
        to[moved] = holes.int()
        ref[holes] = ref[moved]
        ref[moved] = 0
        table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], -one))
    return _returned(st)


def _axis_of(case):
    """Axis of each rotation pair."""
    sec = [int(x) for x in case["sections"].split(",")]
    half, A = case["d"] // 2, len(sec)
    if case["interleaved"]:
        return [i % A if i // A < sec[i % A] else 0 for i in range(half)]
    return [a for a in range(A) for _ in range(sec[a])]


def _plain_axes(st):
    c = st["case"]
    d, hq, hkv = c["d"], c["hq"], c["hkv"]
    q, k, v = _split(st, hq, hkv, d)
    angles = st["positions"].double()[_axis_of(c)].t() * _freqs(d)
    q, k = _rotated(q, st["qw"], angles), _rotated(k, st["kw"], angles)
    st["k"][st["slots"]] = k.bfloat16()
    st["v"][st["slots"]] = v.bfloat16()
    if c["mode"] == "prepare":
        return {"q": q.bfloat16(), "k": st["k"], "v": st["v"]}
    pos = torch.arange(st["max_cached"] + 1, device=DEV)
    slots = (st["base"][:, None] + pos).clamp(max=st["k"].shape[0] - 1)
    see = pos[None, None, :] <= st["lens"].long()[:, None, None]
    o = _attend(q[:, None], st["k"][slots].float(), st["v"][slots].float(), see)
    return {"out": o[:, 0].bfloat16(), "k": st["k"], "v": st["v"]}


# ------------------------------------------------------------------ the framework's calls
def _handle(st):
    """What a user's program sets up once: configuration, cache, workspace, outputs."""
    h = st.get("handle")
    if h is not None:
        return h
    from causal_gqa_attention_qkv_gb300 import attn
    c = st["case"]
    h = {"attn": attn}
    if c["op"] == "cache4":
        h["cfg"] = attn.config(c["hq"], c["hkv"], c["d"], EPS, THETA)
        h["kv"] = attn.KVCache(st["k"], st["v"], st["base"], st["lens"], st["cap"], st["table"], c["page"], K_SCALE,
                               V_SCALE, k_block_scale=st["ks"], v_block_scale=st["vs"])
        n = st["qkv"].shape[0]
        h["ws"] = attn.new_workspace(h["cfg"], n, st["lens"].numel(), st["max_len"])
        h["out"] = torch.empty(n, c["hq"] * c["d"], dtype=torch.bfloat16, device=DEV)
        h["k_new"] = torch.empty(n, c["hkv"], c["d"], dtype=torch.bfloat16, device=DEV)
        h["v_new"] = torch.empty_like(h["k_new"])
    elif c["op"] == "pages":
        h["cfg"] = attn.config(c["hkv"], c["hkv"], c["d"], EPS, THETA)
        zero = torch.zeros(1, dtype=torch.int32, device=DEV)
        table = st["table"] if "table" in st else zero.view(1, 1)
        lens = st["lens"] if "lens" in st else zero
        h["kv"] = attn.KVCache(st["k"], st["v"], torch.zeros(1, dtype=torch.int64, device=DEV), lens, lens, table,
                               c["page"], k_block_scale=st.get("ks"), v_block_scale=st.get("vs"))
        h["ws"] = attn.new_pages_workspace(h["kv"])
    else:
        h["cfg"] = attn.config(c["hq"], c["hkv"], c["d"], EPS, THETA)
        h["kv"] = attn.KVCache(st["k"], st["v"], st["base"], st["lens"], st["cap"])
        n = c["tokens"]
        sec = [int(x) for x in c["sections"].split(",")]
        h["rope"] = attn.RopeAxes(st["positions"], sec, c["interleaved"])
        if c["mode"] == "prepare":
            h["ws"] = attn.new_workspace(h["cfg"], 0, 1, 1)
        else:
            h["ws"] = attn.new_workspace(h["cfg"], n, n, st["max_cached"] + 1)
            h["out"] = torch.empty(n, c["hq"] * c["d"], dtype=torch.bfloat16, device=DEV)
    st["handle"] = h
    return h


def _own(st):
    h = _handle(st)
    attn, cfg, kv, ws, c = h["attn"], h["cfg"], h["kv"], h["ws"], st["case"]
    if c["op"] == "cache4":
        if c["mode"] == "decode":
            attn.decode(cfg, st["qkv"], st["qw"], st["kw"], st["max_cached"], kv, h["out"], ws)
        else:
            attn.prefill(cfg, st["qkv"], st["qw"], st["kw"], st["cu"], st["max_new"], kv, h["out"], ws)
        attn.kv_gather(cfg, kv, st["cu"], st["lens"], h["k_new"], h["v_new"], ws)
        return {"out": h["out"], "k_new": h["k_new"], "v_new": h["v_new"]}
    if c["op"] == "pages":
        st["now"].copy_(st["start"])
        if c["mode"] == "copy":
            attn.pages_copy(cfg, kv, st["src"], st["dst"], ws)
        elif c["mode"] == "fork":
            attn.pages_fork(cfg, kv, st["ref"], st["src"], st["dst"], ws)
        elif c["mode"] == "turnover":
            attn.pages_free(kv, st["ref"], st["ended"], ws)
            attn.pages_reserve(kv, st["ref"], st["grow"], st["more"], ws)
        else:
            attn.pages_compact(cfg, kv, st["ref"], ws)
        return _returned(st)
    if c["mode"] == "prepare":
        attn.prefill_prepare(cfg, st["qkv"], st["qw"], st["kw"], st["cu"], kv, st["q"], ws, rope=h["rope"])
        return {"q": st["q"], "k": st["k"], "v": st["v"]}
    attn.decode(cfg, st["qkv"], st["qw"], st["kw"], st["max_cached"], kv, h["out"], ws, rope=h["rope"])
    return {"out": h["out"], "k": st["k"], "v": st["v"]}


def run(state):
    if own:
        return _own(state)
    return {"cache4": _plain_cache4, "pages": _plain_pages, "axes": _plain_axes}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definitions in 64 bits
def _norm64(x, w):
    x = x.double()
    return w.double() * x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)


def _turn64(x, place):
    """Rotate-half of x [H, N, D] with pair i of token t at place[t, i]."""
    h = x.shape[-1] // 2
    i = torch.arange(h, device=x.device, dtype=torch.float64)
    a = place.double() / torch.exp(i * (math.log(THETA) * 2 / x.shape[-1]))
    return torch.cat((x[..., :h] * torch.cos(a) - x[..., h:] * torch.sin(a),
                      x[..., h:] * torch.cos(a) + x[..., :h] * torch.sin(a)), -1)


def _nearest(x, grid):
    """The nearest of the sorted values `grid`; of two equally near the one at an even index."""
    hi = torch.searchsorted(grid, x).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    a, b = x - grid[lo], grid[hi] - x
    return torch.where((a < b) | ((a == b) & (lo % 2 == 0)), grid[lo], grid[hi])


def _stored64(x, scale):
    """The values that a four-bit cache holds for x [..., D] in 64 bits."""
    half = torch.arange(127, device=x.device)
    e, m = half // 8, half % 8
    e4m3 = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.double() - 10))
    e2m1 = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    y = (x / scale).unflatten(-1, (-1, 16))
    s = _nearest(y.abs().amax(-1, keepdim=True) / 6, e4m3)
    z = torch.where(s > 0, y / s, torch.zeros_like(y))
    return (torch.sign(z) * _nearest(z.abs(), e2m1) * s).flatten(-2) * scale


def _read64(codes, scales, scale):
    mag = torch.tensor(E2M1, dtype=torch.float64, device=codes.device)
    n = torch.stack((codes % 16, codes // 16), -1).flatten(-2).long()
    v = mag[n % 8] * (1 - 2 * (n // 8)).double()
    return (v.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).double()[..., None]).flatten(-2) * scale


def _rows64(q, k, v, first):
    """Causal attention in 64 bits: q [Hq, n, D] at places first .., k and v [Hkv, L, D]."""
    g = q.shape[0] // k.shape[0]
    out = torch.empty_like(q)
    for h in range(k.shape[0]):
        s = q[h * g:(h + 1) * g] @ k[h].t() / math.sqrt(q.shape[-1])
        hidden = torch.arange(k.shape[1], device=q.device)[None] > first + torch.arange(q.shape[1], device=q.device)[:, None]
        out[h * g:(h + 1) * g] = torch.softmax(s.masked_fill(hidden, -math.inf), -1) @ v[h]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "pages":
        return None
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    x = st["qkv"].view(-1, hq + 2 * hkv, d).transpose(0, 1)
    if case["op"] == "axes":
        place = torch.stack([st["positions"][a] for a in _axis_of(case)], -1)
    else:
        place = st["pos"][:, None].expand(-1, d // 2)
    q = _turn64(_norm64(x[:hq], st["qw"]), place)
    k = _turn64(_norm64(x[hq:hq + hkv], st["kw"]), place)
    v = x[hq + hkv:].double()
    if case["op"] == "axes":
        # a cache's entry is its 16-bit value: the attention reads those
        st["k"][st["slots"]] = k.transpose(0, 1).bfloat16()
        st["v"][st["slots"]] = v.transpose(0, 1).bfloat16()
        kk, vv = st["k"].double(), st["v"].double()
        kk[st["slots"]] = k.transpose(0, 1)
        if case["mode"] == "prepare":
            return {"q": q.transpose(0, 1), "k": kk, "v": vv}
        out = []
        for b in range(case["tokens"]):
            at, n = int(st["base"][b]), int(st["lens"][b]) + 1
            o = _rows64(q[:, b:b + 1], st["k"][at:at + n].double().transpose(0, 1),
                        st["v"][at:at + n].double().transpose(0, 1), n - 1)
            out.append(o.reshape(-1))
        return {"out": torch.stack(out), "k": kk, "v": vv}
    kq, vq = _stored64(k, K_SCALE), _stored64(v, V_SCALE)
    out = []
    for b in range(st["lens"].numel()):
        t0, t1, c = int(st["cu"][b]), int(st["cu"][b + 1]), int(st["lens"][b])
        p = torch.arange(c, device=DEV)
        slots = st["table"][b].long()[p // case["page"]] * case["page"] + p % case["page"] if case["page"] else st["base"][b] + p
        kk = _read64(st["k"][slots].transpose(0, 1), st["ks"][:, slots], K_SCALE)
        vv = _read64(st["v"][slots].transpose(0, 1), st["vs"][:, slots], V_SCALE)
        o = _rows64(q[:, t0:t1], torch.cat((kk, kq[:, t0:t1]), 1), torch.cat((vv, vq[:, t0:t1]), 1), c)
        out.append(o.transpose(0, 1).reshape(t1 - t0, -1))
    return {"out": torch.cat(out), "k_new": kq.transpose(0, 1), "v_new": vq.transpose(0, 1)}
