"""GPU tests of the page calls: every result (tables, counts, lengths, contents
of every page) is held to a plain list-and-dict form of the definitions, for
all cache types, at sizes where a rank crosses a warp, a CTA or the cluster,
and for each refusal; then a serving loop of reserve, append, fork, decode,
free and compact against caches that were never shared or moved."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_gqa_attention_qkv_gb300 import build
    build.build()


class Pool:
    """A pool with random contents and requests of the given cached lengths,
    pages drawn at random."""

    def __init__(self, kind, P, ps, hkv, d, lens, rows, ppr, seed=0, extra_slots=0):
        from causal_gqa_attention_qkv_gb300 import attn
        g = torch.Generator().manual_seed(seed)
        self.P, self.ps, self.kind = P, ps, kind
        S = P * ps + extra_slots
        w = {"bf16": 2 * d, "e4m3": d, "e2m1": d // 2}[kind]
        raw = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8).cuda()
        k, v = raw(S, hkv, w), raw(S, hkv, w)
        blocks = [raw(hkv, S, d // 16) for _ in range(2)] if kind == "e2m1" else [None, None]
        if kind == "bf16":
            k, v = k.view(torch.bfloat16), v.view(torch.bfloat16)
        self.cfg = attn.config(hkv, hkv, d)
        perm = torch.randperm(P, generator=g).int()
        table = torch.full((rows, ppr), -1, dtype=torch.int32)
        at = 0
        for b, c in enumerate(lens):
            n = -(-c // ps)
            table[b, :n] = perm[at:at + n]
            at += n
        ref = torch.zeros(P, dtype=torch.int32)
        ref[perm[:at].long()] = 1
        cl = torch.zeros(rows, dtype=torch.int32)
        cl[:len(lens)] = torch.tensor(lens, dtype=torch.int32)
        cap = torch.full((rows,), ppr * ps, dtype=torch.int32, device="cuda")
        self.kv = attn.KVCache(k, v, torch.zeros(rows, dtype=torch.int64, device="cuda"), cl.cuda(), cap, table.cuda(),
                               ps, 0.03, 0.06, *blocks)
        self.ref = ref.cuda()
        self.ws = attn.new_pages_workspace(self.kv)

    def pages(self):
        """Contents by page: [P, bytes] of each array."""
        n = self.P * self.ps
        out = [t[:n].contiguous().view(torch.uint8).view(self.P, -1).cpu() for t in (self.kv.k_cache, self.kv.v_cache)]
        for t in (self.kv.k_block_scale, self.kv.v_block_scale):
            if t is not None:
                out.append(t[:, :n].reshape(t.shape[0], self.P, -1).transpose(0, 1).reshape(self.P, -1).cpu())
        return out

    def state(self):
        return [self.kv.page_table.cpu(), self.ref.cpu(), self.kv.cache_lens.cpu()] + self.pages()

    def status(self):
        from causal_gqa_attention_qkv_gb300 import attn
        return attn.get_status(self.ws)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def same(a, b):
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


# ------------------------------------------------------------------ plain forms
def plain_reserve(st, ps, rows, more):
    table, ref, lens = st[0], st[1], st[2]
    free = [p for p in range(len(ref)) if ref[p] == 0]
    want = []
    for b, m in zip(rows, more):
        c = int(lens[b])
        want += [(b, e) for e in range(-(-c // ps), -(-(c + m) // ps)) if table[b, e] == -1]
    if len(want) > len(free):
        return False
    for (b, e), p in zip(want, free):
        table[b, e] = p
        ref[p] = 1
    return True


def plain_fork(st, ps, src, dst, sb):
    table, ref, lens, pages = st[0], st[1], st[2], st[3:]
    free = [p for p in range(len(ref)) if ref[p] == 0]
    if sum(int(lens[s]) % ps != 0 for s in src) > len(free):
        return False
    for s, t in zip(src, dst):
        c = int(lens[s])
        table[t] = -1
        table[t, :c // ps] = table[s, :c // ps]
        for e in range(c // ps):
            ref[table[s, e]] += 1
        if c % ps:
            p, old = free.pop(0), int(table[s, c // ps])
            table[t, c // ps] = p
            ref[p] = 1
            for i, x in enumerate(pages):
                if i < 2:  # entries: the first c % ps slots
                    n = x.shape[1] // ps * (c % ps)
                    x[p, :n] = x[old, :n]
                else:  # block scales [Hkv, ps, D/16] of a page
                    v = x.view(x.shape[0], -1, ps, sb)
                    v[p, :, :c % ps] = v[old, :, :c % ps]
        lens[t] = c
    return True


def plain_free(st, rows):
    table, ref, lens = st[0], st[1], st[2]
    for b in rows:
        for p in table[b][table[b] >= 0].tolist():
            ref[p] -= 1
        table[b] = -1
        lens[b] = 0


def plain_compact(st):
    table, ref, pages = st[0], st[1], st[3:]
    used = [p for p in range(len(ref)) if ref[p] > 0]
    L = len(used)
    to = dict(zip([p for p in used if p >= L], [h for h in range(L) if ref[h] == 0]))
    for p, h in to.items():
        ref[h], ref[p] = int(ref[p]), 0
        for x in pages:
            x[h] = x[p]
    where = torch.arange(len(ref), dtype=torch.int32)
    for p, h in to.items():
        where[p] = h
    table.copy_(torch.where(table >= 0, where[table.clamp(min=0).long()], table))


KINDS = ["bf16", "e4m3", "e2m1"]


# ------------------------------------------------------------------ one call
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("P,ps,hkv,d,lens,ways,extra", [
    (40, 64, 2, 64, [100, 64, 1, 0, 320], 2, 0),
    (700, 64, 3, 128, [63, 65, 128, 1000, 5000], 3, 5),       # a pool that ends inside a page
    (300, 128, 1, 128, [129, 127, 2000], 1, 0),
    (9000, 64, 1, 64, list(range(1, 2000, 97)), 4, 0),        # ranks across CTAs of the plan
])
def test_fork(kind, P, ps, hkv, d, lens, ways, extra):
    from causal_gqa_attention_qkv_gb300 import attn
    n = len(lens)
    pool = Pool(kind, P, ps, hkv, d, lens, n * (1 + ways) + 2, -(-max(lens) // ps) + 1, seed=P + d, extra_slots=extra)
    src = [b for b in range(n) for _ in range(ways)]
    dst = list(range(n + 1, n + 1 + len(src)))[::-1]
    st = pool.state()
    assert plain_fork(st, ps, src, dst, d // 16)
    attn.pages_fork(pool.cfg, pool.kv, pool.ref, i32(src), i32(dst), pool.ws)
    assert pool.status() == 0
    same(pool.state(), st)


@pytest.mark.parametrize("P,rows,seed", [(1, 1, 0), (31, 3, 1), (33, 2, 2), (256, 7, 3), (5000, 60, 4), (70001, 300, 5)])
def test_reserve_free_reserve(P, rows, seed):
    from causal_gqa_attention_qkv_gb300 import attn
    rng = np.random.RandomState(seed)
    ps = 64
    each = max(1, P // rows // 2)
    lens = [int(rng.randint(0, each * ps + 1)) for _ in range(rows)] if P > 1 else [0]
    while sum(-(-c // ps) for c in lens) > P:
        lens[int(np.argmax(lens))] = 0
    pool = Pool("bf16", P, ps, 1, 64, lens, rows, 2 * each + 3, seed=seed)
    st = pool.state()
    for turn in range(3):
        pick = rng.permutation(rows)[:max(1, rows // 2)].tolist()
        more = [int(rng.randint(0, 3 * ps)) for _ in pick]
        more = [min(m, (2 * each + 3) * ps - int(st[2][b])) for m, b in zip(more, pick)]
        ok = plain_reserve(st, ps, pick, more)
        attn.pages_reserve(pool.kv, pool.ref, i32(pick), i32(more), pool.ws)
        assert pool.status() == (0 if ok else attn.ATTN_STATUS_PAGES)
        same(pool.state()[:3], st[:3])
        gone = rng.permutation(rows)[:max(1, rows // 4)].tolist()
        plain_free(st, gone)
        attn.pages_free(pool.kv, pool.ref, i32(gone), pool.ws)
        assert pool.status() == 0
        same(pool.state(), st)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("P,ps,hkv,d,lens", [
    (50, 64, 2, 128, [300, 64, 700, 1]),
    (1000, 64, 1, 64, [500] * 60),
    (130, 128, 3, 64, [0]),                                   # nothing in use
    (20, 64, 1, 64, [64] * 20),                               # everything in use
    (64, 64, 1, 128, [64] * 31 + [65]),
    (20000, 64, 1, 64, [600] * 900),
])
def test_compact(kind, P, ps, hkv, d, lens):
    from causal_gqa_attention_qkv_gb300 import attn
    rows = len(lens) + 2
    pool = Pool(kind, P, ps, hkv, d, lens, rows, -(-max(lens + [1]) // ps) + 1, seed=P, extra_slots=7 if P == 50 else 0)
    if len(lens) > 3:  # shared pages
        pool.kv.page_table[len(lens), 0] = pool.kv.page_table[0, 0]
        pool.ref[pool.kv.page_table[0, 0].long()] += 1
    st = pool.state()
    for _ in range(2):  # the second call finds nothing to move
        plain_compact(st)
        attn.pages_compact(pool.cfg, pool.kv, pool.ref, pool.ws)
        assert pool.status() == 0
        same(pool.state(), st)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("P,ps,hkv,d,n", [(2, 64, 1, 64, 1), (300, 64, 5, 128, 90), (40, 256, 8, 128, 20)])
def test_copy(kind, P, ps, hkv, d, n):
    from causal_gqa_attention_qkv_gb300 import attn
    pool = Pool(kind, P, ps, hkv, d, [0], 1, 1, seed=n, extra_slots=3)
    perm = torch.randperm(P, generator=torch.Generator().manual_seed(n)).tolist()
    src, dst = perm[:n], perm[n:2 * n]
    src[-1] = src[0]  # one page may be read twice
    st = pool.state()
    for x in st[3:]:
        x[dst] = x[src]
    attn.pages_copy(pool.cfg, pool.kv, i32(src), i32(dst), pool.ws)
    assert pool.status() == 0
    same(pool.state(), st)
    attn.pages_copy(pool.cfg, pool.kv, i32([0, -1, P, 0]), i32([0, 0, 0, P]), pool.ws)  # onto itself; not in the pool
    assert pool.status() == attn.ATTN_STATUS_PAGES
    same(pool.state(), st)


# ------------------------------------------------------------------ refusals that the device sees
def test_refused_calls_change_nothing():
    from causal_gqa_attention_qkv_gb300 import attn
    pool = Pool("e2m1", 12, 64, 1, 64, [100, 130, 64, 5], 8, 4, seed=3)  # 2 + 3 + 1 + 1 pages: 5 are free
    st = pool.state()
    bad_fork = [([0], [1]), ([0], [8]), ([0], [-1]), ([8], [4]), ([-3], [4]), ([0, 1], [4, 4]), ([0, 4], [4, 5])]
    for src, dst in bad_fork:
        attn.pages_fork(pool.cfg, pool.kv, pool.ref, i32(src), i32(dst), pool.ws)
        assert pool.status() == attn.ATTN_STATUS_PAGES, (src, dst)
        same(pool.state(), st)
    bad_reserve = [([8], [1]), ([-1], [1]), ([0, 0], [1, 1]), ([0], [-1]), ([0], [200]), ([4, 5], [256, 100]),
                   ([0, 1], [0, 1000])]
    for rows, more in bad_reserve:
        attn.pages_reserve(pool.kv, pool.ref, i32(rows), i32(more), pool.ws)
        assert pool.status() == attn.ATTN_STATUS_PAGES, (rows, more)
        same(pool.state(), st)
    attn.pages_reserve(pool.kv, pool.ref, i32([4]), i32([256]), pool.ws)  # 4 of the 5 left: fits
    assert pool.status() == 0
    st = pool.state()
    attn.pages_fork(pool.cfg, pool.kv, pool.ref, i32([0, 1]), i32([5, 6]), pool.ws)  # 2 wanted, 1 free
    assert pool.status() == attn.ATTN_STATUS_PAGES
    same(pool.state(), st)
    # a source whose table does not hold what its length says
    pool.kv.cache_lens[3] = 100
    st = pool.state()
    attn.pages_fork(pool.cfg, pool.kv, pool.ref, i32([3]), i32([6]), pool.ws)
    assert pool.status() == attn.ATTN_STATUS_PAGES
    same(pool.state(), st)


def test_free_of_bad_rows_and_entries():
    from causal_gqa_attention_qkv_gb300 import attn
    pool = Pool("bf16", 20, 64, 1, 64, [300, 100, 64], 4, 6, seed=5)
    pool.kv.page_table[0, 4] = 1 << 20
    pool.kv.page_table[1, 5] = 77
    st = pool.state()
    attn.pages_free(pool.kv, pool.ref, i32([9, -1]), pool.ws)
    assert pool.status() == attn.ATTN_STATUS_PAGES
    same(pool.state(), st)
    attn.pages_free(pool.kv, pool.ref, i32([2, 2, 2]), pool.ws)  # emptied once
    assert pool.status() == 0
    attn.pages_free(pool.kv, pool.ref, i32([0, 1]), pool.ws)
    assert pool.status() == attn.ATTN_STATUS_PAGES
    table, ref, lens = pool.state()[:3]
    assert (table == -1).all() and (lens == 0).all()
    assert int(ref.sum()) == 1 and (ref >= 0).all()  # the page that its row no longer listed


def test_empty_lists_are_no_ops():
    from causal_gqa_attention_qkv_gb300 import attn
    pool = Pool("bf16", 5, 64, 1, 64, [70], 2, 2)
    st, none = pool.state(), i32([])
    attn.pages_reserve(pool.kv, pool.ref, none, none, pool.ws)
    attn.pages_fork(pool.cfg, pool.kv, pool.ref, none, none, pool.ws)
    attn.pages_free(pool.kv, pool.ref, none, pool.ws)
    attn.pages_copy(pool.cfg, pool.kv, none, none, pool.ws)
    assert pool.status() == 0
    same(pool.state(), st)


def test_calls_replayed_from_a_graph_and_on_another_stream():
    """fork + free + reserve + compact recorded once and replayed from the same
    start: the eager result each time."""
    from causal_gqa_attention_qkv_gb300 import attn
    pool = Pool("e2m1", 400, 64, 2, 128, [500, 77, 640, 3], 12, 12, seed=8)
    src, dst, gone, grow, more = i32([0, 1, 1, 3]), i32([4, 5, 6, 7]), i32([0, 6]), i32([4, 8, 1]), i32([70, 129, 1])
    names = ("k_cache", "v_cache", "k_block_scale", "v_block_scale", "page_table", "cache_lens")
    start = {n: getattr(pool.kv, n).clone() for n in names} | {"ref": pool.ref.clone()}

    def restore():
        for n in names:
            getattr(pool.kv, n).copy_(start[n])
        pool.ref.copy_(start["ref"])

    def calls():
        attn.pages_fork(pool.cfg, pool.kv, pool.ref, src, dst, pool.ws)
        attn.pages_free(pool.kv, pool.ref, gone, pool.ws)
        attn.pages_reserve(pool.kv, pool.ref, grow, more, pool.ws)
        attn.pages_compact(pool.cfg, pool.kv, pool.ref, pool.ws)

    calls()
    assert pool.status() == 0
    want = pool.state()
    restore()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls()
    s.synchronize()
    same(pool.state(), want)
    g = torch.cuda.CUDAGraph()
    restore()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        calls()
    for _ in range(3):
        restore()
        g.replay()
        torch.cuda.synchronize()
        same(pool.state(), want)


# ------------------------------------------------------------------ all of it together
@pytest.mark.parametrize("kind,axes", [("bf16", False), ("e2m1", True), ("e4m3", False), ("e2m1", False)])
def test_serving_loop(kind, axes):
    """Prompts are prefilled into reserved pages, forked, decoded for some steps
    with pages reserved as they go, some end, the pool is compacted, the others
    go on.  Every output is compared bit for bit with the same requests each
    alone in a contiguous cache."""
    from causal_gqa_attention_qkv_gb300 import attn
    hq, hkv, d, ps, P, rows, ppr = 8, 2, 128, 64, 60, 10, 6
    pool = Pool(kind, P, ps, hkv, d, [], rows, ppr, seed=4)
    cfg, kv, ref, ws = attn.config(hq, hkv, d), pool.kv, pool.ref, pool.ws
    W = (hq + 2 * hkv) * d
    g = torch.Generator().manual_seed(11)
    qw, kw = [(1 + 0.1 * torch.randn(d, generator=g)).bfloat16().cuda() for _ in range(2)]
    aws = attn.new_workspace(cfg, 512, rows, ppr * ps)
    sections = [24, 20, 20]

    def rope_of(pos):  # axes that differ: time, half of it, a third of it
        p = torch.tensor(list(pos), dtype=torch.int32)
        return attn.RopeAxes(torch.stack((p, p // 2, p // 3)).cuda(), sections, True) if axes else None

    class Alone:
        """One request in a contiguous cache of its own."""

        def __init__(self, other=None):
            S = ppr * ps
            w = {"bf16": 2 * d, "e4m3": d, "e2m1": d // 2}[kind]
            raw = torch.zeros(2, S, hkv, w, dtype=torch.uint8, device="cuda")
            k, v = (raw[0].view(torch.bfloat16), raw[1].view(torch.bfloat16)) if kind == "bf16" else raw
            b = [None] * 2
            if kind == "e2m1":
                b = [torch.zeros(hkv, S, d // 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
            self.kv = attn.KVCache(k, v, torch.zeros(1, dtype=torch.int64, device="cuda"), i32([0]), i32([S]), None, 0,
                                   0.03, 0.06, *b)
            self.n = 0
            if other is not None:
                for name in ("k_cache", "v_cache", "k_block_scale", "v_block_scale", "cache_lens"):
                    if getattr(other.kv, name) is not None:
                        getattr(self.kv, name).copy_(getattr(other.kv, name))
                self.n = other.n

        def prefill(self, qkv):
            out = torch.empty(qkv.shape[0], hq * d, dtype=torch.bfloat16, device="cuda")
            attn.prefill(cfg, qkv, qw, kw, i32([0, qkv.shape[0]]), qkv.shape[0], self.kv, out, aws,
                         rope=rope_of(range(self.n, self.n + qkv.shape[0])))
            self.grow(qkv.shape[0])
            return out

        def decode(self, qkv):
            out = torch.empty(1, hq * d, dtype=torch.bfloat16, device="cuda")
            attn.decode(cfg, qkv, qw, kw, 255, self.kv, out, aws, rope=rope_of([self.n]))
            self.grow(1)
            return out

        def grow(self, n):
            self.n += n
            self.kv.cache_lens += n

    new = lambda n: torch.randn(n, W, generator=g).bfloat16().cuda()
    prompts = {0: new(100), 1: new(64), 2: new(130)}
    alone = {}
    attn.pages_reserve(kv, ref, i32([0, 1, 2]), i32([100, 64, 130]), ws)
    cu = [0, 100, 164, 294]
    out = torch.empty(294, hq * d, dtype=torch.bfloat16, device="cuda")
    attn.prefill(cfg, torch.cat([prompts[b] for b in range(3)]), qw, kw, i32(cu), 130, kv.rows(0, 3), out, aws,
                 rope=rope_of([*range(100), *range(64), *range(130)]))
    kv.cache_lens[:3] += i32([100, 64, 130])
    for b in range(3):
        alone[b] = Alone()
        assert torch.equal(alone[b].prefill(prompts[b]).view(torch.int16), out[cu[b]:cu[b + 1]].view(torch.int16))
    attn.pages_fork(cfg, kv, ref, i32([0, 0, 2]), i32([3, 4, 5]), ws)
    for s, t in ((0, 3), (0, 4), (2, 5)):
        alone[t] = Alone(alone[s])

    def decode_steps(active, steps):
        for _ in range(steps):
            attn.pages_reserve(kv, ref, i32(active), i32([1] * len(active)), ws)
            qkv = new(len(active))
            n = len(active)
            view = attn.KVCache(kv.k_cache, kv.v_cache, kv.slot_base[:n], kv.cache_lens[active], kv.slot_capacity[:n],
                                kv.page_table[active].contiguous(), ps, 0.03, 0.06, kv.k_block_scale, kv.v_block_scale)
            o = torch.empty(n, hq * d, dtype=torch.bfloat16, device="cuda")
            attn.decode(cfg, qkv, qw, kw, 255, view, o, aws, rope=rope_of([alone[b].n for b in active]))
            kv.cache_lens[active] += 1
            for i, b in enumerate(active):
                assert torch.equal(alone[b].decode(qkv[i:i + 1]).view(torch.int16), o[i:i + 1].view(torch.int16)), b

    decode_steps([0, 1, 2, 3, 4, 5], 30)
    attn.pages_free(kv, ref, i32([0, 2]), ws)
    attn.pages_compact(cfg, kv, ref, ws)
    used = int((ref > 0).sum())
    assert (ref[:used] > 0).all() and (ref[used:] == 0).all()
    decode_steps([1, 3, 4, 5], 10)
    attn.pages_fork(cfg, kv, ref, i32([4]), i32([0]), ws)
    alone[0] = Alone(alone[4])
    decode_steps([0, 4, 5], 5)
    attn.pages_free(kv, ref, i32([0, 1, 3, 4, 5]), ws)
    assert (ref == 0).all() and (kv.page_table == -1).all()
    assert attn.get_status(ws) == 0 and attn.get_status(aws) == 0


@pytest.mark.parametrize("kind", ["bf16", "e2m1"])
def test_a_captured_step_of_reserve_and_decode_crosses_pages(kind):
    """Reserve, decode over the pool's own rows and the lengths' increment, recorded
    once: replayed across page boundaries right behind a fork and a free, every
    output equals the one over contiguous caches bit for bit."""
    from causal_gqa_attention_qkv_gb300 import attn
    hq, hkv, d, ps, rows, ppr, steps = 4, 2, 128, 64, 4, 5, 140
    pool = Pool(kind, 24, ps, hkv, d, [], rows, ppr, seed=6)
    cfg, kv, ws = attn.config(hq, hkv, d), pool.kv, pool.ws
    W, S = (hq + 2 * hkv) * d, ppr * ps
    g = torch.Generator().manual_seed(12)
    qw, kw = [(1 + 0.1 * torch.randn(d, generator=g)).bfloat16().cuda() for _ in range(2)]
    new = lambda n: torch.randn(n, W, generator=g).bfloat16().cuda()
    aws = attn.new_workspace(cfg, 256, rows, S)
    lens = [63, 100, 0, 0]
    blocks = [None, None]
    if kind == "e2m1":
        blocks = [torch.zeros(hkv, rows * S, d // 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
    like = lambda t: torch.zeros(rows * S, *t.shape[1:], dtype=torch.uint8, device="cuda").view(t.dtype) \
        if t.dtype == torch.uint8 else torch.zeros(rows * S, *t.shape[1:], dtype=t.dtype, device="cuda")
    flat = attn.KVCache(like(kv.k_cache), like(kv.v_cache), torch.arange(0, rows * S, S, device="cuda"),
                        torch.zeros(rows, dtype=torch.int32, device="cuda"), kv.slot_capacity.clone(), None, 0, 0.03,
                        0.06, *blocks)
    prompts = new(163)
    cu = i32([0, 63, 163])
    attn.pages_reserve(kv, pool.ref, i32([0, 1]), i32([63, 100]), ws)
    for c in (kv, flat):
        out = torch.empty(163, hq * d, dtype=torch.bfloat16, device="cuda")
        attn.prefill(cfg, prompts, qw, kw, cu, 100, c.rows(0, 2), out, aws)
        c.cache_lens[:2] += i32([63, 100])
    for s, t in ((0, 2), (1, 3)):  # what the fork below does, by copies
        flat.k_cache[t * S:t * S + S] = flat.k_cache[s * S:s * S + S]
        flat.v_cache[t * S:t * S + S] = flat.v_cache[s * S:s * S + S]
        for b in blocks:
            if b is not None:
                b[:, t * S:t * S + S] = b[:, s * S:s * S + S].clone()
        flat.cache_lens[t] = flat.cache_lens[s]
    every, ones = i32(list(range(rows))), i32([1] * rows)
    qkv, out = new(rows), torch.empty(rows, hq * d, dtype=torch.bfloat16, device="cuda")
    attn.pages_fork(cfg, kv, pool.ref, i32([0, 1]), i32([2, 3]), ws)

    def step():
        attn.pages_reserve(kv, pool.ref, every, ones, ws)
        attn.decode(cfg, qkv, qw, kw, S - 1, kv, out, aws)
        kv.cache_lens.add_(1)

    step()  # eager, straight behind the fork
    want = torch.empty_like(out)
    attn.decode(cfg, qkv, qw, kw, S - 1, flat, want, aws)
    flat.cache_lens.add_(1)
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        qkv.copy_(new(rows))
        if i == steps // 2:  # two requests end, another is forked into their place
            attn.pages_free(kv, pool.ref, i32([2, 3]), ws)
            attn.pages_fork(cfg, kv, pool.ref, i32([1, 0]), i32([2, 3]), ws)
            for s, t in ((1, 2), (0, 3)):
                flat.k_cache[t * S:t * S + S] = flat.k_cache[s * S:s * S + S]
                flat.v_cache[t * S:t * S + S] = flat.v_cache[s * S:s * S + S]
                for b in blocks:
                    if b is not None:
                        b[:, t * S:t * S + S] = b[:, s * S:s * S + S].clone()
                flat.cache_lens[t] = flat.cache_lens[s]
        graph.replay()
        attn.decode(cfg, qkv, qw, kw, S - 1, flat, want, aws)
        flat.cache_lens.add_(1)
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)), i
    assert torch.equal(kv.cache_lens, flat.cache_lens)
    assert attn.get_status(ws) == 0 and attn.get_status(aws) == 0


def test_two_pools_on_two_streams_at_once():
    """Calls on different pools, each with its own workspace, do not meet."""
    from causal_gqa_attention_qkv_gb300 import attn
    make = lambda seed: Pool("e2m1", 300, 64, 2, 128, [500, 77, 640, 3], 12, 12, seed=seed)

    def calls(pool):
        attn.pages_fork(pool.cfg, pool.kv, pool.ref, lists[0], lists[1], pool.ws)
        attn.pages_free(pool.kv, pool.ref, lists[2], pool.ws)
        attn.pages_reserve(pool.kv, pool.ref, lists[3], lists[4], pool.ws)
        attn.pages_compact(pool.cfg, pool.kv, pool.ref, pool.ws)

    lists = [i32(x) for x in ([0, 1, 1, 3], [4, 5, 6, 7], [0, 6], [4, 8, 1], [70, 129, 1])]
    want = []
    for seed in (21, 22):
        pool = make(seed)
        calls(pool)
        want.append(pool.state())
    pools, streams = [make(21), make(22)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for pool, s in zip(pools, streams):
        with torch.cuda.stream(s):
            calls(pool)
    torch.cuda.synchronize()
    for pool, w in zip(pools, want):
        assert pool.status() == 0
        same(pool.state(), w)


def test_lists_longer_than_the_plan_has_warps_or_lanes():
    """Several list entries per warp (more than 32 of them too), a row that asks
    for more than 32 pages, runs of pages of more than one look, a refusal that only
    the last row causes, and a list of every row in reverse."""
    from causal_gqa_attention_qkv_gb300 import attn
    ps, P, rows, ppr = 64, 40000, 9000, 45
    rng = np.random.RandomState(9)
    lens = [int(x) for x in rng.randint(0, 2 * ps, rows)]
    pool = Pool("bf16", P, ps, 1, 64, lens, rows, ppr, seed=9)
    st = pool.state()
    rows_list = list(range(rows))[::-1]
    more = [int(x) for x in rng.randint(0, 2 * ps, rows)]
    for b in (0, 17, 4444, 8999):
        more[rows_list.index(b)] = 40 * ps
    free = P - int((st[1] > 0).sum())
    need = sum(-(-(lens[b] + m) // ps) - -(-lens[b] // ps) for b, m in zip(rows_list, more))
    assert need < free
    over = more[:-1] + [ppr * ps - lens[0] + 1]  # the last row's length would not fit its table
    attn.pages_reserve(pool.kv, pool.ref, i32(rows_list), i32(over), pool.ws)
    assert pool.status() == attn.ATTN_STATUS_PAGES
    same(pool.state()[:3], st[:3])
    assert plain_reserve(st, ps, rows_list, more)
    attn.pages_reserve(pool.kv, pool.ref, i32(rows_list), i32(more), pool.ws)
    assert pool.status() == 0
    same(pool.state()[:3], st[:3])
    gone = rng.permutation(rows)[:4000].tolist()
    plain_free(st, gone)
    attn.pages_free(pool.kv, pool.ref, i32(gone), pool.ws)
    src = [b for b in range(rows) if b not in set(gone)][:1200]  # five forks per warp
    assert plain_fork(st, ps, src, gone[:1200], 4)
    attn.pages_fork(pool.cfg, pool.kv, pool.ref, i32(src), i32(gone[:1200]), pool.ws)
    assert pool.status() == 0
    same(pool.state(), st)
    plain_compact(st)
    attn.pages_compact(pool.cfg, pool.kv, pool.ref, pool.ws)
    assert pool.status() == 0
    same(pool.state(), st)


@pytest.mark.parametrize("kind", ["e2m1", "bf16"])
def test_offsets_past_32_bits(kind):
    """The same request in the first and in the last pages of a pool of more than
    2^32 bytes: the same bits from prefill, decode and gather, after a copy and a
    fork between the two ends too."""
    from causal_gqa_attention_qkv_gb300 import attn
    hq, hkv, d, ps, ppr = 8, 8, 128, 64, 4
    w = {"bf16": 2 * d, "e2m1": d // 2}[kind]
    P = (1 << 32) // (ps * hkv * w) + 9
    S = P * ps
    k, v = [torch.empty(S, hkv, w, dtype=torch.uint8, device="cuda") for _ in range(2)]
    blocks = [torch.empty(hkv, S, d // 16, dtype=torch.uint8, device="cuda") for _ in range(2)] if kind == "e2m1" else [None] * 2
    if kind == "bf16":
        k, v = k.view(torch.bfloat16), v.view(torch.bfloat16)
    table = [[2, 0, 1, -1], [P - 1, P - 3, P - 2, -1], [-1] * 4]
    kv = attn.KVCache(k, v, torch.zeros(3, dtype=torch.int64, device="cuda"), i32([0, 0, 0]), i32([ppr * ps] * 3), i32(table),
                      ps, 0.03, 0.06, *blocks)
    ref = torch.zeros(P, dtype=torch.int32, device="cuda")
    ref[[0, 1, 2, P - 1, P - 2, P - 3]] = 1
    ref[3:P - 3] = 1  # taken by others, but for the page that the fork below gets
    ref[P - 5] = 0
    cfg, ws, n = attn.config(hq, hkv, d), attn.new_pages_workspace(kv), 150
    aws = attn.new_workspace(cfg, 2 * n, 3, ppr * ps)
    g = torch.Generator().manual_seed(3)
    nw = [(1 + 0.1 * torch.randn(d, generator=g)).bfloat16().cuda() for _ in range(2)]
    x = torch.randn(n + 1, (hq + 2 * hkv) * d, generator=g).bfloat16().cuda()
    new = lambda m: torch.empty(m, hq * d, dtype=torch.bfloat16, device="cuda")
    same_rows = lambda t: all(torch.equal(t[0].view(torch.int16), r.view(torch.int16)) for r in t[1:])
    out = new(2 * n)
    attn.prefill(cfg, torch.cat([x[:n], x[:n]]), *nw, i32([0, n, 2 * n]), n, kv.rows(0, 2), out, aws)
    assert same_rows(out.view(2, n, -1)) and torch.isfinite(out).all()
    kv.cache_lens[:2] += n
    attn.pages_fork(cfg, kv, ref, i32([0]), i32([2]), ws)  # its open page is page 1, the copy page P - 5
    assert kv.page_table[2].tolist() == [2, 0, P - 5, -1]
    dec = new(3)
    attn.decode(cfg, x[n:].expand(3, -1).contiguous(), *nw, ppr * ps - 1, kv, dec, aws)
    assert same_rows(dec) and torch.isfinite(dec).all()
    kv.cache_lens += 1
    ko, vo = [torch.empty(3 * (n + 1), hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    attn.kv_gather(cfg, kv, i32([0, n + 1, 2 * n + 2, 3 * n + 3]), i32([0, 0, 0]), ko, vo, aws)
    assert same_rows(ko.view(3, n + 1, -1)) and same_rows(vo.view(3, n + 1, -1))
    attn.pages_copy(cfg, kv, i32([2, 0]), i32([P - 7, P - 6]), ws)
    kv.page_table[0, :2] = i32([P - 7, P - 6])
    k2, v2 = torch.empty_like(ko), torch.empty_like(vo)
    attn.kv_gather(cfg, kv, i32([0, n + 1, 2 * n + 2, 3 * n + 3]), i32([0, 0, 0]), k2, v2, aws)
    assert torch.equal(ko.view(torch.int16), k2.view(torch.int16)) and torch.equal(vo.view(torch.int16), v2.view(torch.int16))
    assert attn.get_status(ws) == 0 and attn.get_status(aws) == 0
