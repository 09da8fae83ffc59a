"""Cases of the operators for long caches and constrained sampling: attention
over the blocks of a cache that a cheap score selects for each query (bounds of
a block's keys, selection, attention over the selected blocks), and the rules
that logits go through before a token is drawn (penalties for tokens that a
request has seen, biases, grammar masks) with the table of seen tokens.

A case names an operator ("op") with sizes.  ``run`` computes it in plain torch
operations, or with ``own`` through the framework's calls.  ``exact`` gives the
values of the definitions in 64 bits.

A block is ``block`` consecutive positions of a request.  Its bounds are the
lowest and the highest entry of its keys in each component, per KV head, kept
for full blocks.  The query of a token at position p sees blocks 0 .. p / block;
its KV head's list holds all of them where they are no more than ``keep``, else
the ``first`` first, the ``last`` last and, of the others, those with the largest
  sum over the group's heads h and components d of max(q_hd lo_d, q_hd hi_d)
(ties: the lower block), in ascending order, -1 behind them.

Seen tokens: one 16-bit word per token of the vocabulary and row, bit 15 set if
the token is in the prompt, the rest the number of times it was generated.
Logits: x + bias, then x / r or x r (x > 0 or not) for seen tokens, then
x - frequency * count and x - presence for generated ones, then -inf where the
row's grammar mask has no bit.
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


# ------------------------------------------------------------------ cases
def _bounds(name, kind, batch, lo, hi, new, hkv, d, page, block, again):
    return {"name": name, "op": "bounds", "type": kind, "batch": batch, "lo": lo, "hi": hi, "new": new, "hkv": hkv,
            "d": d, "page": page, "block": block, "again": again}


def _select(name, kind, batch, lo, hi, new, hq, hkv, d, page, block, first, last, keep):
    return {"name": name, "op": "select", "type": kind, "batch": batch, "lo": lo, "hi": hi, "new": new, "hq": hq,
            "hkv": hkv, "d": d, "page": page, "block": block, "first": first, "last": last, "keep": keep}


def _attend(name, kind, batch, lo, hi, new, hq, hkv, d, page, block, keep):
    return {"name": name, "op": "attend", "type": kind, "batch": batch, "lo": lo, "hi": hi, "new": new, "hq": hq,
            "hkv": hkv, "d": d, "page": page, "block": block, "keep": keep}


def _seen(name, batch, lo, hi, vocab, prompt):
    return {"name": name, "op": "seen", "batch": batch, "lo": lo, "hi": hi, "vocab": vocab, "prompt": prompt}


def _adjust(name, batch, vocab, history, biases, masked):
    return {"name": name, "op": "adjust", "batch": batch, "vocab": vocab, "history": history, "biases": biases,
            "masked": masked}


def listed():
    return [
        # a long prompt has just been appended: bounds of all its blocks
        _bounds("bounds prompt", "bf16", 1, 0, 0, 32768, 8, 128, 64, 64, False),
        # chunks of prompts over a four-bit cache, odd lengths, larger blocks and
        # pages, bounds made anew from the start of each request (as after a move of its pages)
        _bounds("bounds four-bit anew", "e2m1", 9, 333, 9000, 300, 4, 128, 256, 128, True),
        # one user's next token over a long document: the latency of a call
        _select("select one", "bf16", 1, 65000, 65000, 1, 32, 8, 128, 64, 64, 1, 4, 64),
        # a batch's next tokens, cached lengths from short (all blocks) to long
        _select("select batch", "e4m3", 64, 500, 16384, 1, 32, 8, 128, 64, 64, 1, 2, 32),
        # a few drafted tokens per request, contiguous regions
        _select("select drafts", "bf16", 12, 20001, 100000, 8, 64, 8, 128, 0, 64, 2, 3, 48),
        # one user's next token: few heads, the keys split over the card
        _attend("attend one", "bf16", 1, 65000, 65000, 1, 32, 8, 128, 64, 64, 64),
        # a batch's next tokens, 4096 keys each
        _attend("attend batch", "bf16", 64, 5000, 16384, 1, 32, 8, 128, 64, 64, 64),
        # chunks of prompts over an eight-bit cache, small heads, odd lengths
        _attend("attend chunk", "e4m3", 3, 3001, 9000, 200, 16, 2, 64, 64, 64, 24),
        # new requests take their rows: prompts of up to 8192 tokens marked
        _seen("seen prompts", 64, 100, 8192, 151936, True),
        # the tokens of a step counted
        _seen("seen step", 96, 1, 1, 32003, False),
        # the benchmark's sampling batch with every rule
        _adjust("adjust batch", 64, 151936, 3000, 300, True),
        # one request, penalties only
        _adjust("adjust one", 1, 32003, 500, 0, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("bounds", "select", "select", "attend", "attend", "seen", "adjust", "adjust"))
    hq, hkv, d = rng.choice(((32, 8, 128), (16, 2, 64), (8, 8, 128), (64, 8, 128), (8, 4, 64), (6, 3, 128), (4, 1, 128)))
    kind, block = rng.choice(("bf16", "bf16", "e4m3", "e2m1")), rng.choice((64, 64, 128, 256))
    page = rng.choice((0, block, max(block, 128), 256))
    if op == "seen":
        prompt = rng.random() < 0.6
        vocab = _log(rng, 1000, 120000)
        hi = _log(rng, 2, min(6000, vocab // 2)) if prompt else 1
        c = _seen("", _log(rng, 1, 64), rng.randint(1, hi), hi, vocab, prompt)
    elif op == "adjust":
        vocab = _log(rng, 100, 150000)
        c = _adjust("", _log(rng, 1, 60), vocab, _log(rng, 1, 4000), rng.choice((0, 1, _log(rng, 2, 400))),
                    rng.random() < 0.5)
    elif op == "bounds":
        batch, again = _log(rng, 1, 40), rng.random() < 0.5
        hi = _log(rng, 2 * block, max(1000, 60000 // batch))  # some block becomes full
        new = _log(rng, 1 if again else block, max(300, 30000 // batch))
        c = _bounds("", kind, batch, rng.randint(0, hi), hi, new, hkv, d, page, block, again)
    else:
        drafts = rng.random() < 0.3
        batch = _log(rng, 1, 8 if drafts else 60)
        new = _log(rng, 2, 40) if drafts else 1
        hi = _log(rng, 14 * block, min(100000, 600000 // batch))
        lo = rng.randint(hi // 20, hi)
        keep = _log(rng, 4, 64)
        if op == "select":  # the longest request has something to choose
            first, last = rng.randint(0, 2), rng.randint(1, 2)
            keep = min(max(keep, first + last + 2), hi // block // 2)
            c = _select("", kind, batch, lo, hi, new, hq, hkv, d, page, block, first, last, keep)
        else:
            keep = max(1, keep * 64 // block)
            c = _attend("", kind, batch, lo, hi, new, hq, hkv, d, page, block, keep)
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
    return _spread(case["lo"], case["hi"], B), _spread(max(1, case["new"] // 3), case["new"], B)


def _entry_bytes(kind, d):
    return {"bf16": 2 * d, "e4m3": d, "e2m1": d // 2 + d // 16}[kind]


def work(case):
    if case["op"] == "seen":
        n = sum(_spread(case["lo"], case["hi"], case["batch"]))
        table = 2 * case["batch"] * case["vocab"]
        # a prompt's row is emptied first; a step reads and writes a word per token, its table is given back whole
        return {"bytes": 4 * n + (table if case["prompt"] else 2 * table), "flops": 0}
    if case["op"] == "adjust":
        n = case["batch"] * case["vocab"]
        return {"bytes": n * (4 + 4 + 2) + (n // 8 if case["masked"] else 0) + 8 * case["batch"] * case["biases"],
                "flops": 4.0 * n}
    cached, new = _lens(case)
    d, hkv, bs = case["d"], case["hkv"], case["block"]
    if case["op"] == "bounds":
        full = sum((c + n) // bs - (0 if case["again"] else c // bs) for c, n in zip(cached, new))
        return {"bytes": full * hkv * (bs * _entry_bytes(case["type"], d) + 4 * d), "flops": 2.0 * full * bs * hkv * d}
    hq, keep, N = case["hq"], case["keep"], sum(new)
    if case["op"] == "select":
        seen = sum((c + n - 1) // bs for c, n in zip(cached, new) if (c + n - 1) // bs + 1 > keep)
        flops = sum(4.0 * hkv * d * ((c + j) // bs) for c, n in zip(cached, new) for j in range(n))
        return {"bytes": seen * hkv * 4 * d + N * (hq * d * 2 + hkv * keep * 4), "flops": flops}
    # what the lists of a request's tokens reach at least: one token's keys
    reach = sum(min(c + n, keep * bs) for c, n in zip(cached, new))
    keys = sum(min(c + j + 1, keep * bs) for c, n in zip(cached, new) for j in range(n))
    return {"bytes": 2 * reach * hkv * _entry_bytes(case["type"], d) + N * (2 * hq * d * 2 + hkv * keep * 4),
            "flops": 4.0 * keys * hq * d}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _randint(g, lo, hi, shape, dtype=torch.int64):
    return torch.randint(lo, hi, shape, generator=g, device=DEV, dtype=dtype)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _layout(case, g, st):
    """Requests, their cached and new lengths, and where their entries lie."""
    cached, new = _lens(case)
    B, page = len(cached), case["page"]
    full = [c + n for c, n in zip(cached, new)]
    st.update(max_len=max(full), max_new=max(new), lens=_i32(cached),
              cu=_i32([sum(new[:b]) for b in range(B + 1)]), one=max(new) == 1,
              req=torch.tensor([b for b in range(B) for _ in range(new[b])], device=DEV),
              pos=torch.tensor([cached[b] + j for b in range(B) for j in range(new[b])], device=DEV))
    if page:
        need = [-(-n // page) for n in full]
        total, ppr = sum(need) + 3, max(need)
        perm = torch.randperm(total, generator=g, device=DEV).int()
        at = torch.tensor([sum(need[:b]) for b in range(B)], device=DEV)[:, None] + torch.arange(ppr, device=DEV)
        live = torch.arange(ppr, device=DEV) < torch.tensor(need, device=DEV)[:, None]
        st["table"] = torch.where(live, perm[at.clamp(max=total - 1)], torch.full_like(perm[:1], -1)).contiguous()
        st["base"] = torch.zeros(B, dtype=torch.int64, device=DEV)
        st["cap"] = torch.full((B,), ppr * page, dtype=torch.int32, device=DEV)
        st["slots"] = total * page
        st["rows"], st["row_base"] = st["slots"] // case["block"], None
    else:
        st["table"] = None
        starts = [3 + sum(full[:b]) + 3 * b for b in range(B)]
        blocks = [-(-n // case["block"]) for n in full]
        st["base"] = torch.tensor(starts, device=DEV)
        st["cap"] = _i32(full)
        st["slots"] = starts[-1] + full[-1] + 3
        st["row_base"] = torch.tensor([sum(blocks[:b]) + b for b in range(B)], device=DEV)
        st["rows"] = sum(blocks) + B


def _entries(case, g, st, name):
    """A pool of entries: codes take every finite value, a few bits of range for the scales."""
    kind, d, shape = case["type"], case["d"], (st["slots"], case["hkv"])
    st[name + "s"] = None
    if kind == "bf16":
        st[name] = torch.empty(*shape, d, dtype=torch.bfloat16, device=DEV)
        for part in st[name].split(1 << 18):
            part.copy_(_randn(g, *part.shape))
    elif kind == "e4m3":
        st[name] = _randint(g, 0, 2, (*shape, d), torch.uint8).mul_(128).add_(_randint(g, 0, 113, (*shape, d), torch.uint8))
    else:
        st[name] = _randint(g, 0, 256, (*shape, d // 2), torch.uint8)
        st[name + "s"] = _randint(g, 56, 90, (case["hkv"], st["slots"], d // 16), torch.uint8)


def _prepare_bounds(case, g):
    st = {"case": case}
    _layout(case, g, st)
    _entries(case, g, st, "k")
    st["v"], st["vs"] = st["k"], st["ks"]  # V has no part in it
    st["bounds"] = torch.zeros(st["rows"], case["hkv"], 2, case["d"], dtype=torch.bfloat16, device=DEV)
    st["start"] = torch.zeros_like(st["lens"]) if case["again"] else st["lens"]
    return st


def _queries(case, g, n):
    q = _randn(g, n, case["hq"], case["d"])
    return q.bfloat16() if case["type"] == "bf16" else q.half()


def _prepare_select(case, g):
    st = {"case": case}
    _layout(case, g, st)
    w = {"bf16": case["d"], "e4m3": case["d"], "e2m1": case["d"] // 2}[case["type"]]
    t = torch.bfloat16 if case["type"] == "bf16" else torch.uint8
    # the cache is there, but selection does not read it
    st["k"] = torch.empty(st["slots"], case["hkv"], w, dtype=t, device=DEV)
    st["ks"] = None
    if case["type"] == "e2m1":
        st["ks"] = torch.empty(case["hkv"], st["slots"], case["d"] // 16, dtype=torch.uint8, device=DEV)
    st["v"], st["vs"] = st["k"], st["ks"]
    shape = (st["rows"], case["hkv"], case["d"])
    mid, half = 0.7 * _randn(g, *shape), 1.6 + 0.3 * _randn(g, *shape)
    st["bounds"] = torch.stack((mid - half.abs(), mid + half.abs()), 2).bfloat16()
    del mid, half
    st["q"] = _queries(case, g, st["req"].numel())
    st["list"] = torch.empty(st["req"].numel(), case["hkv"], case["keep"], dtype=torch.int32, device=DEV)
    return st


def _prepare_attend(case, g):
    st = {"case": case}
    _layout(case, g, st)
    _entries(case, g, st, "k")
    _entries(case, g, st, "v")
    n, keep, bs = st["req"].numel(), case["keep"], case["block"]
    st["q"] = _queries(case, g, n)
    # lists as a selection leaves them: the first and the last block, others at random, ascending
    most = -(-st["max_len"] // bs)
    last = (st["pos"] // bs)[:, None, None]
    j = torch.arange(most, device=DEV)
    score = torch.rand(n, case["hkv"], most, generator=g, device=DEV)
    score = torch.where((j == 0) | (j == last), score + 1, score).masked_fill(j > last, -1.0)
    best, at = score.topk(min(keep, most), -1)
    at = torch.where(best >= 0, at, torch.full_like(at, 1 << 30)).sort(-1).values
    st["list"] = torch.full((n, case["hkv"], keep), -1, dtype=torch.int32, device=DEV)
    st["list"][..., :at.shape[-1]] = torch.where(at < 1 << 30, at, torch.full_like(at, -1)).int()
    return st


def _tokens(g, n, vocab):
    """Tokens as texts have them: low numbers far more often than high ones."""
    u = torch.rand(n, generator=g, device=DEV)
    return (vocab * u * u * u).long().clamp(max=vocab - 1).int()


def _prepare_seen(case, g):
    B, V = case["batch"], case["vocab"]
    new = _spread(case["lo"], case["hi"], B)
    st = {"case": case, "cu": _i32([sum(new[:b]) for b in range(B + 1)]), "tokens": _tokens(g, sum(new), V),
          "req": torch.tensor([b for b in range(B) for _ in range(new[b])], device=DEV)}
    # requests sit in rows of a larger table, in no order
    st["rows"] = torch.randperm(B, generator=g, device=DEV).int()
    ld = -(-V // 8) * 8
    st["start"] = torch.zeros(B, ld, dtype=torch.int16, device=DEV)
    st["start"][:, :V] = _randint(g, 0, 50, (B, V), torch.int16).clamp_(min=46).sub_(46)
    st["seen"] = st["start"].clone()
    return st


def _prepare_adjust(case, g):
    B, V, n = case["batch"], case["vocab"], case["biases"]
    ld = -(-V // 8) * 8
    st = {"case": case, "logits": 3 * _randn(g, B, V)}
    seen = torch.zeros(B, ld, dtype=torch.int32, device=DEV)
    rows = torch.arange(B, device=DEV).repeat_interleave(case["history"])
    out = _tokens(g, rows.numel(), V).long()
    seen.index_put_((rows, out), torch.ones_like(out, dtype=torch.int32), accumulate=True)
    prompt = _tokens(g, rows.numel(), V).long()
    seen[rows, prompt] |= 0x8000
    st["seen"] = torch.where(seen >= 0x8000, seen - 0x10000, seen).short()
    st["rows"] = torch.randperm(B, generator=g, device=DEV).int()
    st["repetition"] = 1 + 0.5 * torch.rand(B, generator=g, device=DEV)
    st["presence"] = torch.rand(B, generator=g, device=DEV) - 0.2
    st["frequency"] = 0.5 * torch.rand(B, generator=g, device=DEV)
    st["bias_start"] = _i32([n * b for b in range(B + 1)])
    st["bias_row"] = torch.arange(B, device=DEV).repeat_interleave(n)
    n = min(n, V)
    st["bias_token"] = torch.cat([torch.randperm(V, generator=g, device=DEV)[:case["biases"]] if n == case["biases"] else
                                  _randint(g, 0, V, (case["biases"],)) for _ in range(B)]).int()
    st["bias_value"] = 4 * _randn(g, B * case["biases"])
    words = -(-V // 32)
    # grammars allow few tokens: a tenth of them here
    bits = torch.rand(B, words, 32, generator=g, device=DEV) < 0.1
    st["mask"] = (bits.long() << torch.arange(32, device=DEV)).sum(-1).int()
    st["mask_rows"] = torch.randperm(B, generator=g, device=DEV).int()
    st["out"] = torch.empty_like(st["logits"])
    return st


def prepare(case, seed):
    return {"bounds": _prepare_bounds, "select": _prepare_select, "attend": _prepare_attend, "seen": _prepare_seen,
            "adjust": _prepare_adjust}[case["op"]](case, _gen(seed))


# ------------------------------------------------------------------ plain forms
def _read(st, name, slots, heads=slice(None)):
    """fp32 entries of slots (and KV heads): [..., D], with all heads [..., Hkv, D]."""
    kind, scale = st["case"]["type"], K_SCALE if name == "k" else V_SCALE
    x = st[name][slots, heads]
    if kind == "bf16":
        return x.float()
    if kind == "e4m3":
        return x.view(torch.float8_e4m3fn).float() * scale
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    v = torch.stack((table[(x & 15).int()], table[(x >> 4).int()]), -1).unflatten(-2, (-1, 8)).flatten(-2)
    s = st[name + "s"].transpose(0, 1)[slots, heads].view(torch.float8_e4m3fn).float()
    return (v * s[..., None]).flatten(-2) * scale


def _slots(st, req, pos):
    """Slots of the positions pos of the requests req (broadcast)."""
    page = st["case"]["page"]
    if page:
        return st["table"].long()[req, (pos // page).clamp(max=st["table"].shape[1] - 1)].clamp(min=0) * page + pos % page
    return (st["base"][req] + pos).clamp(max=st["slots"] - 1)


def _rows(st, req, blk):
    """Rows of the bounds of blocks blk of the requests req."""
    if st["row_base"] is not None:
        return (st["row_base"][req] + blk).clamp(max=st["rows"] - 1)
    return _slots(st, req, blk * st["case"]["block"]) // st["case"]["block"]


def _plain_bounds(st):
    bs = st["case"]["block"]
    lens, cu = st["lens"].long(), st["cu"].long()
    lo, hi = st["start"].long() // bs, (lens + cu[1:] - cu[:-1]) // bs
    j = torch.arange(-(-st["max_len"] // bs), device=DEV)
    req, blk = ((j >= lo[:, None]) & (j < hi[:, None])).nonzero().unbind(1)
    for r, b in zip(req.split(1024), blk.split(1024)):
        x = _read(st, "k", _slots(st, r[:, None], b[:, None] * bs + torch.arange(bs, device=DEV)))
        st["bounds"][_rows(st, r, b)] = torch.stack((x.amin(1), x.amax(1)), 2).bfloat16()
    return st["bounds"]


def _plain_select(st):
    c = st["case"]
    bs, keep, hkv, d = c["block"], c["keep"], c["hkv"], c["d"]
    j = torch.arange(-(-st["max_len"] // bs), device=DEV)
    B = st["lens"].numel()
    rows = _rows(st, torch.arange(B, device=DEV)[:, None], j)
    out = []
    for req, pos, q in zip(st["req"].split(16), st["pos"].split(16), st["q"].split(16)):
        # scores next to the border decide: 64 bits
        x = q.double().view(-1, hkv, c["hq"] // hkv, d)
        a = torch.stack((x.clamp(max=0).sum(2), x.clamp(min=0).sum(2)), 2)  # times lo, times hi
        b = st["bounds"][rows[req]].flatten(3).transpose(1, 2).double()
        s = torch.matmul(b, a.flatten(2)[..., None])[..., 0]  # [n, Hkv, blocks]
        del b
        last = (pos // bs)[:, None, None]
        s = torch.where((j < c["first"]) | (j > last - c["last"]), torch.full_like(s, math.inf), s)
        s = s.masked_fill(j > last, -math.inf)
        at = s.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
        at = torch.where(at <= last, at, torch.full_like(at, 1 << 30)).sort(-1).values
        r = torch.full((q.shape[0], hkv, keep), -1, dtype=torch.int32, device=DEV)
        r[..., :at.shape[-1]] = torch.where(at < 1 << 30, at, torch.full_like(at, -1)).int()
        out.append(r)
    return torch.cat(out)


def _plain_attend(st):
    c = st["case"]
    bs, keep, hkv, d = c["block"], c["keep"], c["hkv"], c["d"]
    heads = torch.arange(hkv, device=DEV)[:, None]
    step = max(1, (1 << 28) // (hkv * keep * bs * d))
    out = []
    for req, pos, q, ls in zip(*(t.split(step) for t in (st["req"], st["pos"], st["q"], st["list"]))):
        at = (ls.long()[..., None] * bs + torch.arange(bs, device=DEV)).flatten(2)  # [n, Hkv, keys]
        see = (at >= 0) & (at <= pos[:, None, None])
        slots = _slots(st, req[:, None, None], at.clamp(min=0))
        k, v = _read(st, "k", slots, heads), _read(st, "v", slots, heads)
        x = q.float().view(-1, hkv, c["hq"] // hkv, d)
        s = torch.matmul(x, k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
        s = s.masked_fill(~see[:, :, None], -math.inf)
        p = torch.exp(s - s.amax(-1, keepdim=True))
        o = torch.matmul(p / p.sum(-1, keepdim=True), v)
        out.append(o.flatten(1).bfloat16())
        del k, v
    return torch.cat(out)


def _plain_seen(st):
    c = st["case"]
    row, tok = st["rows"].long()[st["req"]], st["tokens"].long()
    seen = st["seen"]
    if c["prompt"]:
        seen[st["rows"].long()] = 0
        seen[row, tok] |= -32768
        return seen
    seen.copy_(st["start"])
    words = seen.int() & 0xFFFF
    add = torch.zeros_like(words)
    add.index_put_((row, tok), torch.ones_like(tok, dtype=torch.int32), accumulate=True)
    words = (words & 0x8000) | ((words & 0x7FFF) + add).clamp(max=0x7FFF)
    seen.copy_(torch.where(words >= 0x8000, words - 0x10000, words).short())
    return seen


def _plain_adjust(st):
    c = st["case"]
    V = c["vocab"]
    x = st["logits"]
    if c["biases"]:
        x = x.index_put((st["bias_row"], st["bias_token"].long()), st["bias_value"], accumulate=True)
    w = st["seen"][st["rows"].long(), :V].int() & 0xFFFF
    r = st["repetition"][:, None]
    x = torch.where(w != 0, torch.where(x > 0, x / r, x * r), x)
    n = w & 0x7FFF
    x = x - st["frequency"][:, None] * n.float()
    x = x - st["presence"][:, None] * (n > 0).float()
    if c["masked"]:
        m = st["mask"][st["mask_rows"].long()]
        bits = ((m[..., None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1).flatten(1)[:, :V]
        x = x.masked_fill(bits == 0, -math.inf)
    return x


# ------------------------------------------------------------------ the framework's calls
def _handle(st):
    """What a user's program sets up once: configuration, cache, workspace, outputs."""
    h = st.get("handle")
    if h is not None:
        return h
    from causal_gqa_attention_qkv_gb300 import attn
    c = st["case"]
    h = {"attn": attn}
    if c["op"] == "adjust":
        h["rules"] = attn.LogitsRules(
            seen=st["seen"], seen_row=st["rows"], repetition=st["repetition"], presence=st["presence"],
            frequency=st["frequency"], bias_start=st["bias_start"] if c["biases"] else None,
            bias_token=st["bias_token"] if c["biases"] else None, bias_value=st["bias_value"] if c["biases"] else None,
            mask=st["mask"] if c["masked"] else None, mask_row=st["mask_rows"] if c["masked"] else None)
    elif c["op"] != "seen":
        h["cfg"] = attn.config(c.get("hq", c["hkv"]), c["hkv"], c["d"], EPS, THETA)
        scales = {} if c["type"] == "bf16" else {"k_scale": K_SCALE, "v_scale": V_SCALE}
        h["kv"] = attn.KVCache(st["k"], st["v"], st["base"], st["lens"], st["cap"], st["table"], c["page"], **scales,
                               k_block_scale=st["ks"], v_block_scale=st["vs"])
        if "bounds" in st:
            h["blocks"] = attn.BlockBounds(st["bounds"], c["block"], st["row_base"])
        n = st["req"].numel()
        h["cu"] = None if st["one"] else st["cu"]
        h["ws"] = attn.new_block_workspace(h["cfg"], n, st["max_len"], c["block"], c.get("keep", 1))
        if c["op"] == "attend":
            h["out"] = torch.empty(n, c["hq"] * c["d"], dtype=torch.bfloat16, device=DEV)
    st["handle"] = h
    return h


def _own(st):
    h, c = _handle(st), st["case"]
    attn = h["attn"]
    if c["op"] == "bounds":
        attn.block_bounds(h["cfg"], h["kv"], h["blocks"], h["cu"], h["ws"], start=st["start"] if c["again"] else None)
        return st["bounds"]
    if c["op"] == "select":
        attn.block_select(h["cfg"], st["q"], h["cu"], st["max_len"], h["kv"], h["blocks"], c["first"], c["last"],
                          st["list"], h["ws"])
        return st["list"]
    if c["op"] == "attend":
        attn.block_attend(h["cfg"], st["q"], h["cu"], h["kv"], c["block"], st["list"], h["out"], h["ws"])
        return h["out"]
    if c["op"] == "seen":
        if c["prompt"]:
            attn.tokens_seen(st["seen"], c["vocab"], st["rows"], st["tokens"], st["cu"], prompt=True, clear=True)
        else:
            st["seen"].copy_(st["start"])
            attn.tokens_seen(st["seen"], c["vocab"], st["rows"], st["tokens"])
        return st["seen"]
    return attn.logits_adjust(st["logits"], h["rules"], out=st["out"])


def run(state):
    if own:
        return _own(state)
    return {"bounds": _plain_bounds, "select": _plain_select, "attend": _plain_attend, "seen": _plain_seen,
            "adjust": _plain_adjust}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definitions in 64 bits
def _values64(st, name, where, head):
    """Entries [len(where), D] of one KV head in 64 bits."""
    kind, raw = st["case"]["type"], st[name][where, head]
    if kind == "bf16":
        return raw.double()
    scale = K_SCALE if name == "k" else V_SCALE
    if kind == "e4m3":
        code = raw.long()
        e, m = (code >> 3) & 15, code & 7
        mag = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.double() - 10))
        return torch.where(code >= 128, -mag, mag) * scale
    n = torch.stack((raw % 16, raw // 16), -1).flatten(-2).long()
    mag = torch.tensor(E2M1, dtype=torch.float64, device=DEV)[n % 8] * (1 - 2 * (n // 8)).double()
    s = st[name + "s"][head, where].view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
    return mag * s * scale


def _places(st, b, pos):
    """Slots of the positions pos of request b."""
    page = st["case"]["page"]
    if not page:
        return st["base"][b] + pos
    return st["table"][b, pos // page].long() * page + pos % page


def _exact_bounds(st):
    bs, res = st["case"]["block"], st["bounds"].double()
    for b in range(st["lens"].numel()):
        end = int(st["lens"][b] + st["cu"][b + 1] - st["cu"][b]) // bs
        begin = int(st["start"][b]) // bs
        if end <= begin:
            continue
        pos = torch.arange(begin * bs, end * bs, device=DEV)
        slots = _places(st, b, pos)
        rows = slots[::bs] // bs if st["row_base"] is None else st["row_base"][b] + torch.arange(begin, end, device=DEV)
        for h in range(st["case"]["hkv"]):
            x = _values64(st, "k", slots, h).unflatten(0, (-1, bs))
            res[rows, h, 0], res[rows, h, 1] = x.min(1).values, x.max(1).values
    return res


def _exact_select(st):
    c = st["case"]
    bs, keep, g = c["block"], c["keep"], c["hq"] // c["hkv"]
    res = torch.full_like(st["list"], -1)
    for t in range(st["req"].numel()):
        b, n = int(st["req"][t]), int(st["pos"][t]) // bs + 1
        if n <= keep:
            res[t, :, :n] = torch.arange(n, device=DEV, dtype=torch.int32)
            continue
        lo, hi = c["first"], n - c["last"]
        blk = torch.arange(lo, hi, device=DEV)
        rows = _places(st, b, blk * bs) // bs if st["row_base"] is None else st["row_base"][b] + blk
        for h in range(c["hkv"]):
            q = st["q"][t, h * g:(h + 1) * g].double()[:, None]
            low, high = st["bounds"][rows, h].double().unbind(1)
            s = torch.maximum(q * low, q * high).sum((0, 2))
            order = sorted(range(hi - lo), key=s.neg().tolist().__getitem__)  # a stable sort
            best = [lo + i for i in order[:keep - c["first"] - c["last"]]]
            res[t, h] = _i32(sorted(list(range(lo)) + best + list(range(hi, n))))
    return res


def _exact_attend(st):
    c = st["case"]
    bs, g, d = c["block"], c["hq"] // c["hkv"], c["d"]
    res = torch.zeros(st["req"].numel(), c["hq"], d, dtype=torch.float64, device=DEV)
    for t in range(st["req"].numel()):
        b, p = int(st["req"][t]), int(st["pos"][t])
        for h in range(c["hkv"]):
            blk = st["list"][t, h]
            pos = (blk[blk >= 0].long()[:, None] * bs + torch.arange(bs, device=DEV)).flatten()
            slots = _places(st, b, pos[pos <= p])
            w = st["q"][t, h * g:(h + 1) * g].double() @ _values64(st, "k", slots, h).t() / math.sqrt(d)
            res[t, h * g:(h + 1) * g] = torch.softmax(w, -1) @ _values64(st, "v", slots, h)
    return res.flatten(1)


def _exact_adjust(st):
    c = st["case"]
    res = []
    for b in range(c["batch"]):
        x = st["logits"][b].double()
        at = st["bias_row"] == b
        if c["biases"]:
            x = x.scatter_add(0, st["bias_token"][at].long(), st["bias_value"][at].double())
        word = st["seen"][st["rows"][b].long(), :c["vocab"]].long() % 65536
        count, known = (word % 32768).double(), word > 0
        r = st["repetition"][b].double()
        x = x * torch.where(known, torch.where(x > 0, 1 / r, r), torch.ones_like(x))
        x = x - count * st["frequency"][b].double() - (count > 0).double() * st["presence"][b].double()
        if c["masked"]:
            i = torch.arange(c["vocab"], device=DEV)
            word = st["mask"][st["mask_rows"][b].long()].long()[i // 32]
            x[(word >> (i % 32)) % 2 == 0] = -math.inf
        res.append(x)
    return torch.stack(res)


def exact(case, seed):
    if case["op"] == "seen":
        return None
    st = prepare(case, seed)
    if case["op"] in ("attend", "select") and st["req"].numel() * case["hkv"] > 3000:
        return None
    return {"bounds": _exact_bounds, "select": _exact_select, "attend": _exact_attend,
            "adjust": _exact_adjust}[case["op"]](st)
