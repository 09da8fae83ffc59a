"""Plain 64-bit forms of the calls of include/blocks.h and include/logits.h, and the
setup that their GPU tests share.  They share no code with the CUDA path and are pinned
by tests/test_blocks_host.py."""
import numpy as np
import torch

import ref64

K_SCALE, V_SCALE = 0.03125, 0.0625


def bf16(x: np.ndarray) -> np.ndarray:
    """Rounded to bf16 (nearest even), as fp64."""
    return torch.tensor(np.asarray(x), dtype=torch.float32).bfloat16().double().numpy()


# ------------------------------------------------------------------ blocks
def row_of(c: dict, b: int, i: int) -> int:
    """Row of the bounds of block i of request b; -1 for a page outside the cache."""
    bs, page = c["block"], c["page"]
    if not page:
        return int(c["row_base"][b]) + i
    pg = int(c["table"][b][i * bs // page])
    return (pg * page + i * bs % page) // bs if 0 <= pg < c["slots"] // page else -1


def slots_of(c: dict, b: int, pos) -> np.ndarray:
    """Slots of positions; -1 for a page outside the cache."""
    pos, page = np.asarray(pos), c["page"]
    if not page:
        return int(c["base"][b]) + pos
    pg = np.asarray(c["table"][b])[pos // page].astype(np.int64)
    return np.where((pg >= 0) & (pg < c["slots"] // page), pg * page + pos % page, -1)


def read(entries: np.ndarray, slots: np.ndarray) -> np.ndarray:
    """Entries [n, Hkv, D] of slots, zeros where there is none."""
    return np.where((slots >= 0)[:, None, None], entries[np.maximum(slots, 0)], 0.0)


def bounds(c: dict, keys: np.ndarray, start=None) -> dict:
    """{row: [Hkv, 2, D]} of the blocks that the call makes."""
    out, bs = {}, c["block"]
    for b, (cached, new) in enumerate(zip(c["cached"], c["new"])):
        first = max(int(start[b]) if start is not None else cached, 0) // bs
        for i in range(first, (cached + new) // bs):
            row = row_of(c, b, i)
            if row < 0 or row >= c["rows"]:
                continue
            k = bf16(read(keys, slots_of(c, b, np.arange(i * bs, (i + 1) * bs))))
            with np.errstate(invalid="ignore"):
                out[row] = np.stack((k.min(0), k.max(0)), 1)
    return out


def score(q: np.ndarray, lo: np.ndarray, hi: np.ndarray) -> np.ndarray:
    """q [G, D], lo and hi [n, D] -> [n]; no number counts as the largest."""
    with np.errstate(invalid="ignore"):
        s = lo @ np.minimum(q, 0).sum(0) + hi @ np.maximum(q, 0).sum(0)
    return np.where(np.isnan(s), np.inf, s)


def select(c: dict, q: np.ndarray, rows_bounds: np.ndarray, first: int, last: int, keep: int) -> np.ndarray:
    """Lists [N, Hkv, keep] for q [N, Hq, D] and bounds [rows, Hkv, 2, D]."""
    N, Hkv = q.shape[0], rows_bounds.shape[1]
    G, bs = q.shape[1] // Hkv, c["block"]
    out = np.full((N, Hkv, keep), -1, np.int32)
    t = 0
    for b, (cached, new) in enumerate(zip(c["cached"], c["new"])):
        for j in range(new):
            n = (cached + j) // bs + 1
            if n <= keep:
                out[t, :, :n] = np.arange(n)
            else:
                cand = np.arange(first, n - last)
                rows = np.array([row_of(c, b, i) for i in cand])
                ok = (rows >= 0) & (rows < rows_bounds.shape[0])
                x = np.where(ok[:, None, None, None], rows_bounds[np.where(ok, rows, 0)], 0.0)
                for h in range(Hkv):
                    s = score(q[t, h * G:(h + 1) * G], x[:, h, 0], x[:, h, 1])
                    best = cand[np.argsort(-s, kind="stable")[:keep - first - last]]
                    out[t, h] = np.sort(np.concatenate((np.arange(first), best, np.arange(n - last, n))))
            t += 1
    return out


def attend(c: dict, q: np.ndarray, lists: np.ndarray, keys: np.ndarray, vals: np.ndarray, codes: bool):
    """(out [N, Hq, D], bound on the kernels' error).

    The prepared Q enters the products as it is.  P is rounded to bf16 with what that leaves as a
    second bf16 (2^-16 of it) or, next to codes, to f16 (2^-11, and 2^-25 absolute below its
    normal range, of weights whose largest is at least 1 before the division by their sum);
    fp32 sums and exp2 stay below 2^-16 of sums of magnitudes; the output is rounded to
    bf16 (2^-8).  A score moves by at most d = 2^-16 sum |q_i k_i| / sqrt(D), a weight by a
    factor within exp(+-2 max d), so
      |out - ref| <= 2^-8 |ref| (1 + small) + (exp(2 max d) - 1 + 2 h + 2^-15) sum p |v| + n 2^-24 max |v|.
    """
    h = 2.0 ** -11 if codes else 2.0 ** -16
    N, Hq, D = q.shape
    Hkv, bs = lists.shape[1], c["block"]
    G = Hq // Hkv
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    t = 0
    for b, (cached, new) in enumerate(zip(c["cached"], c["new"])):
        for j in range(new):
            p = cached + j
            for kh in range(Hkv):
                pos = np.concatenate([np.arange(i * bs, min((i + 1) * bs, p + 1)) for i in lists[t, kh].tolist()
                                      if i >= 0 and i * bs <= p] or [np.zeros(0, np.int64)]).astype(np.int64)
                if len(pos) == 0:
                    continue
                s = slots_of(c, b, pos)
                k, v = read(keys, s)[:, kh], read(vals, s)[:, kh]
                x = q[t, kh * G:(kh + 1) * G]
                sc = x @ k.T / np.sqrt(D)
                d = 2.0 ** -16 * (np.abs(x) @ np.abs(k).T) / np.sqrt(D)
                w = np.exp(sc - sc.max(1, keepdims=True))
                w /= w.sum(1, keepdims=True)
                o = w @ v
                grow = np.exp(2 * d.max(1, keepdims=True)) - 1 + 2 * h + 2.0 ** -15
                out[t, kh * G:(kh + 1) * G] = o
                tol[t, kh * G:(kh + 1) * G] = (2.0 ** -8 * 1.01 * np.abs(o) + grow * 1.01 * (w @ np.abs(v)) +
                                               (len(pos) * 2.0 ** -24 * np.abs(v).max() if codes else 0.0))
            t += 1
    return out, tol


class Cache:
    """A cache with random entries, requests of the given cached and new lengths (the cache
    holds both), and bounds."""

    def __init__(self, kind, hq, hkv, d, cached, new, page, block, seed=0, spare=1, extra_rows=0, extra_slots=0):
        from causal_gqa_attention_qkv_gb300 import attn
        self.kind, self.hq, self.hkv, self.d = kind, hq, hkv, d
        rng = np.random.RandomState(seed)
        g = torch.Generator().manual_seed(seed)
        B, full = len(cached), [c + n for c, n in zip(cached, new)]
        c = {"block": block, "page": page, "cached": list(cached), "new": list(new)}
        table = None
        if page:
            need = [-(-n // page) for n in full]
            total = sum(need) + spare
            perm = rng.permutation(total)
            table = np.full((B, max(max(need), 1)), -1, np.int32)
            for b in range(B):
                at = sum(need[:b])
                table[b, :need[b]] = perm[at:at + need[b]]
            base, cap, slots = np.zeros(B, np.int64), np.full(B, table.shape[1] * page), total * page + extra_slots
            c["rows"] = slots // block + extra_rows
            row_base = None
        else:
            base = np.array([5 + sum(full[:b]) + 7 * b for b in range(B)], np.int64)
            cap, slots = np.array(full), int(base[-1]) + full[-1] + 3
            blocks = [-(-n // block) for n in full]
            row_base = np.array([2 + sum(blocks[:b]) + b for b in range(B)], np.int64)
            c["rows"] = int(row_base[-1]) + blocks[-1] + 1 + extra_rows
        c.update(table=table, base=base, slots=slots, row_base=row_base)
        self.c = c
        w = {"bf16": d, "e4m3": d, "e2m1": d // 2}[kind]
        if kind == "bf16":
            k, v = (torch.randn(slots, hkv, w, generator=g).bfloat16() for _ in range(2))
        elif kind == "e4m3":  # every finite code up to 2^4
            k, v = ((torch.randint(0, 2, (slots, hkv, w), generator=g) * 128 +
                     torch.randint(0, 88, (slots, hkv, w), generator=g)).to(torch.uint8) for _ in range(2))
        else:
            k, v = (torch.randint(0, 256, (slots, hkv, w), generator=g).to(torch.uint8) for _ in range(2))
        scales = [None, None]
        if kind == "e2m1":
            scales = [torch.randint(50, 80, (hkv, slots, d // 16), generator=g).to(torch.uint8) for _ in range(2)]
        self.k, self.v, self.scales = k, v, scales
        i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32).cuda()
        self.cfg = attn.config(hq, hkv, d)
        self.kv = attn.KVCache(k.cuda(), v.cuda(), torch.tensor(base).cuda(), i32(cached), i32(cap),
                               None if table is None else i32(table), page, K_SCALE, V_SCALE,
                               *[None if s is None else s.cuda() for s in scales])
        self.bounds = torch.full((c["rows"], hkv, 2, d), 776.0, dtype=torch.bfloat16).cuda()
        self.blocks = attn.BlockBounds(self.bounds, block, None if row_base is None else torch.tensor(row_base).cuda())
        self.N = sum(new)
        self.cu = i32(np.concatenate(([0], np.cumsum(new))))
        t = torch.bfloat16 if kind == "bf16" else torch.float16
        self.q = torch.randn(self.N, hq, d, generator=g).to(t).cuda()

    def workspace(self, keep, max_len=None):
        from causal_gqa_attention_qkv_gb300 import attn
        m = max(x + n for x, n in zip(self.c["cached"], self.c["new"])) if max_len is None else max_len
        return attn.new_block_workspace(self.cfg, self.N, m, self.c["block"], keep)

    @property
    def max_len(self):
        return max(x + n for x, n in zip(self.c["cached"], self.c["new"]))

    def entries(self, name):
        e = self.kv.k_cache if name == "k" else self.kv.v_cache
        s = self.kv.k_block_scale if name == "k" else self.kv.v_block_scale
        scale = 1.0 if self.kind == "bf16" else (K_SCALE if name == "k" else V_SCALE)
        return ref64.entries(e, self.kind, scale, s)

    def q64(self):
        return self.q.double().cpu().numpy()


# ------------------------------------------------------------------ logits
def adjust(x, seen=None, rep=None, pres=None, freq=None, bias=None, mask=None):
    """One row in fp32 steps as the header states them: x [V] fp32, seen [V] words, bias a list of
    (token, value), mask [V] truth values."""
    f = np.float32
    with np.errstate(all="ignore"):
        x = x.astype(f).copy()
        sums = {}
        for t, v in bias or []:
            if 0 <= t < len(x):
                sums[t] = f(sums.get(t, f(0)) + f(v))
        for t, v in sums.items():
            x[t] = f(x[t] + v)
        if seen is not None:
            w = seen.astype(np.int64) & 0xFFFF
            n = (w & 0x7FFF).astype(f)
            if rep is not None and rep > 0:
                x = np.where(w != 0, np.where(x > 0, x / f(rep), x * f(rep)), x).astype(f)
            if freq is not None:
                x = np.where(n > 0, x - f(freq) * n, x).astype(f)
            if pres is not None:
                x = np.where(n > 0, x - f(pres), x).astype(f)
        if mask is not None:
            x = np.where(mask, x, f(-np.inf)).astype(f)
    return x


def seen_rows(table, vocab, rows, groups, prompt=False, clear=False):
    """The table [rows, ld] of words after a call: groups[b] are the tokens for row rows[b]."""
    t = table.astype(np.int64) & 0xFFFF
    R = t.shape[0]
    if clear:
        for r in rows:
            if 0 <= r < R:
                t[r] = 0
    for r, toks in zip(rows, groups):
        if not 0 <= r < R:
            continue
        for v in toks:
            if 0 <= v < vocab:
                if prompt:
                    t[r, v] |= 0x8000
                elif t[r, v] & 0x7FFF != 0x7FFF:
                    t[r, v] += 1
    return np.where(t >= 0x8000, t - 0x10000, t).astype(np.int16)
