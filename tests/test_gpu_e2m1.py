"""GPU tests of four-bit (E2M1) caches: what an append stores, attention over
it (decode, prefill, mixed, projected), reading entries back, and the same bits
from every way of making the same call.  Stored V is held to the format's own
arithmetic exactly; K (whose fp32 value is off by PAIR_REL of its pair) may
differ where that value sits next to a rounding boundary; outputs are held to
the bound derived in ref64.attend over the entries that the cache holds."""
import numpy as np
import pytest
import torch

import ref64
from causal_gqa_attention_qkv_gb300 import inputs as gen
from parity_util import written_slots

pytestmark = pytest.mark.gpu

KS, VS = 0.03, 0.0625


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_gqa_attention_qkv_gb300 import build
    build.build()


def run(w, host):
    from causal_gqa_attention_qkv_gb300 import step
    ds = step.upload(w, host)
    ds.run()
    torch.cuda.synchronize()
    assert ds.status() == 0
    return ds


def cache_of(ds):
    return ds.kv_prefill or ds.kv_decode


def check_stored(w, host, kv, k64, v64):
    """Codes and block scales of the written slots, and that nothing else changed."""
    slots = written_slots(host)
    rest = np.ones(host["k_cache"].shape[0], bool)
    rest[slots] = False
    for name, x, scale in (("k", k64, host["k_scale"]), ("v", v64, host["v_scale"])):
        codes, blocks = getattr(kv, f"{name}_cache").cpu(), getattr(kv, f"{name}_block_scale").cpu()
        assert torch.equal(codes[rest], host[f"{name}_cache"][rest])
        assert torch.equal(blocks[:, rest], host[f"{name}_block_scale"][:, rest])
        c, s = ref64.unpack(codes[slots]), blocks[:, slots].numpy().transpose(1, 0, 2).astype(np.int64)
        rc, rs = ref64.e2m1_store(x, scale)
        if name == "v":
            assert np.array_equal(s, rs), "V block scales"
            assert np.array_equal(ref64.e2m1_value(c), ref64.e2m1_value(rc)), "V codes"
            continue
        # A fp32 K off by r = PAIR_REL of its pair changes a scale or a code only
        # next to a boundary.  Whatever it chose, the entry it stored is the
        # nearest for a value within that error: no further from K than half the
        # gap of the grid there, (gap / 2) s, or the clamped part (6.4 s at most,
        # since s is at least 15/16 of amax / 6).
        assert np.abs(s - rs).max() <= 1
        sv = ref64.e4m3_values()[s][..., None]
        y = (x / scale).reshape(*s.shape, 16)
        e = np.abs(ref64.e2m1_value(c)).reshape(y.shape)
        half_gap = np.where(e >= 4, 1.0, np.where(e >= 2, 0.5, 0.25))
        pair = (ref64.pair_norm(x) / scale).reshape(y.shape)
        off = np.abs(ref64.e2m1_value(c).reshape(y.shape) * sv - y)
        assert (off <= half_gap * sv + ref64.PAIR_REL * pair + 2.0 ** -23 * np.abs(y)).all()
        assert (ref64.e2m1_value(c) != ref64.e2m1_value(rc)).mean() <= 1e-3


def check_out(w, host, kv, out, axes=None, qkv=None):
    q, _, _ = qkv or ref64.prepared(w, host, axes)
    keys = ref64.entries(kv.k_cache, "e2m1", host["k_scale"], kv.k_block_scale)
    vals = ref64.entries(kv.v_cache, "e2m1", host["v_scale"], kv.v_block_scale)
    ref, tol = ref64.attend(w, host, q, keys, vals)
    got = out.double().cpu().numpy().reshape(ref.shape)
    assert np.isfinite(got).all()
    worst = float((np.abs(got - ref) / np.maximum(tol, 1e-300)).max()) if ref.size else 0.0  # an entry of 0 is exact
    assert worst <= 1.0, f"{worst:.2f} x the derived bound"


DECODE = [
    # (Hq, Hkv, D, cached lens, page size)
    (32, 8, 128, [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 255, 256, 257, 1000, 3000], 0),
    (4, 2, 64, [0, 5, 511, 2047], 0),
    (16, 2, 128, [7, 129, 4000], 64),
    (8, 8, 64, [12, 300, 64, 1], 128),
    (16, 2, 64, [33, 900, 4097], 64),
    (6, 3, 128, [0, 70, 6000], 256),
    (2, 1, 128, [9000], 0),
    (128, 16, 128, [40, 513], 0),
    (32, 4, 64, [4200, 2047, 2048] + list(range(1, 2200, 30)), 64),  # splits of 2048 keys, groups of 8
]


@pytest.mark.parametrize("hq,hkv,d,cache,ps", DECODE)
def test_decode(hq, hkv, d, cache, ps):
    w = gen.custom(f"d4_{hq}_{hkv}_{d}_{ps}", hq, hkv, d, [1] * len(cache), cache, seed=len(cache) + d + ps, decode_from=0)
    host = gen.make_inputs(w, page_size=ps, kv_dtype="e2m1", k_scale=KS, v_scale=VS)
    ds = run(w, host)
    _, k, v = ref64.prepared(w, host)
    check_stored(w, host, ds.kv_decode, k, v)
    check_out(w, host, ds.kv_decode, ds.out)


PREFILL = [
    # (Hq, Hkv, D, new lens, cached lens, page size, decode_from)
    (32, 8, 128, [300, 77, 129, 1], [0, 200, 64, 1000], 0, 4),
    (16, 2, 64, [130, 1, 65, 257], [3, 0, 700, 128], 0, 4),
    (8, 2, 128, [300, 77, 213], [0, 200, 64], 64, 3),
    (8, 8, 64, [200, 31], [64, 0], 128, 2),
    (16, 2, 64, [130, 1, 65], [3, 0, 700], 64, 3),
    (6, 3, 128, [40, 0, 9], [0, 7, 255], 64, 3),
    (16, 4, 128, [100, 64, 1, 1, 1], [50, 0, 10, 700, 0], 0, 2),
]


@pytest.mark.parametrize("hq,hkv,d,lens,cache,ps,df", PREFILL)
def test_prefill_and_mixed(hq, hkv, d, lens, cache, ps, df):
    w = gen.custom(f"p4_{hq}_{hkv}_{d}_{ps}_{df}", hq, hkv, d, lens, cache, seed=sum(lens) + d + ps, decode_from=df)
    host = gen.make_inputs(w, page_size=ps, kv_dtype="e2m1", k_scale=KS, v_scale=VS)
    ds = run(w, host)
    _, k, v = ref64.prepared(w, host)
    check_stored(w, host, cache_of(ds), k, v)
    check_out(w, host, cache_of(ds), ds.out)


@pytest.mark.parametrize("hq,hkv,d,ps", [(16, 8, 128, 0), (8, 8, 64, 64)])
def test_prefill_of_many_short_requests(hq, hkv, d, ps):
    """Several work items per CTA, most of them of one key tile: the warps that
    fetch tiles ahead must not wait for an item that is only handed out once the
    fetched tiles are computed."""
    lens = [1 + (7 * i) % 60 for i in range(160)]
    cache = [(13 * i) % 90 for i in range(160)]
    w = gen.custom(f"short4_{d}", hq, hkv, d, lens, cache, seed=d, decode_from=160)
    host = gen.make_inputs(w, page_size=ps, kv_dtype="e2m1", k_scale=KS, v_scale=VS)
    ds = run(w, host)
    check_out(w, host, ds.kv_prefill, ds.out)


@pytest.mark.parametrize("hq,hkv,d,cache,ps", [
    (32, 8, 128, [0, 5, 63, 64, 700, 3000, 9000], 0),
    (4, 2, 64, [12, 300], 0),
    (16, 2, 128, [7, 129, 4000], 64),
])
def test_decode_equals_append_then_attend_and_static_scratch(hq, hkv, d, cache, ps):
    """attn_decode, attn_kv_append + attn_decode_attend and
    attn_decode_static_scratch give the same bits, output and cache."""
    from causal_gqa_attention_qkv_gb300 import attn, step
    w = gen.custom(f"f4_{hq}_{d}_{ps}", hq, hkv, d, [1] * len(cache), cache, seed=d + ps, decode_from=0)
    host = gen.make_inputs(w, page_size=ps, kv_dtype="e2m1", k_scale=KS, v_scale=VS)
    a = run(w, host)
    b, c = step.upload(w, host), step.upload(w, host)
    cu = torch.arange(len(cache) + 1, dtype=torch.int32, device="cuda")
    attn.kv_append(b.cfg, b.qkv, b.k_norm_w, cu, b.kv_decode, b.workspace)
    attn.decode_attend(b.cfg, b.qkv, b.q_norm_w, b.max_cache_len, b.kv_decode, b.out, b.workspace)
    attn.decode_static_scratch(c.cfg, c.qkv, c.q_norm_w, c.k_norm_w, c.max_cache_len, c.kv_decode, c.out)
    torch.cuda.synchronize()
    assert b.status() == 0
    for x in (b, c):
        assert torch.equal(a.out.view(torch.int16), x.out.view(torch.int16))
        for n in ("k_cache", "v_cache", "k_block_scale", "v_block_scale"):
            assert torch.equal(getattr(a.kv_decode, n), getattr(x.kv_decode, n)), n


@pytest.mark.parametrize("d,lens,cache", [(128, [130, 40], [70, 0]), (64, [1, 300], [513, 5])])
def test_paged_equals_contiguous(d, lens, cache):
    w = gen.custom(f"pc4_{d}", 8, 2, d, lens, cache, seed=d)
    a = run(w, gen.make_inputs(w, kv_dtype="e2m1", k_scale=KS, v_scale=VS))
    b = run(w, gen.make_inputs(w, page_size=64, kv_dtype="e2m1", k_scale=KS, v_scale=VS))
    assert torch.equal(a.out.view(torch.int16), b.out.view(torch.int16))


def values_for_borders(d):
    """Rows of V whose entries sit on the format's rounding boundaries: block
    maxima on E4M3 ties and their neighbours, entries on every E2M1 tie, zeros,
    tiny and huge blocks, both signs."""
    t = ref64.e4m3_values()
    amax = 6 * np.concatenate([(t[1:] + t[:-1]) / 2, t[1:]])
    rng = np.random.RandomState(0)
    rows = []
    for a in amax:
        x = rng.choice([0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6], 16) * rng.choice([-1, 1], 16) * a / 6
        x[rng.randint(16)] = a
        rows.append(x)
    rows += [np.zeros(16), np.full(16, -0.0), np.full(16, 2.0 ** -12), np.full(16, 1e30), np.linspace(-4000, 4000, 16)]
    x = np.concatenate(rows)
    x = np.concatenate([x, np.zeros(-len(x) % (2 * d))]).reshape(-1, 2, d)
    return torch.from_numpy(x.astype(np.float32)).bfloat16()


@pytest.mark.parametrize("d", [64, 128])
def test_appended_values_on_the_rounding_boundaries(d):
    """V of crafted values, appended by the prologue and by decode."""
    from causal_gqa_attention_qkv_gb300 import attn, step
    v = values_for_borders(d)
    n = v.shape[0]
    w = gen.custom(f"b4_{d}", 4, 2, d, [n], [0], seed=d)
    host = gen.make_inputs(w, kv_dtype="e2m1", k_scale=KS, v_scale=VS)
    host["qkv"].view(n, 8, d)[:, 6:] = v * VS  # a power of two: exact
    ds = step.upload(w, host)
    attn.kv_append(ds.cfg, ds.qkv, ds.k_norm_w, ds.cu_seqlens, ds.kv_prefill, ds.workspace)
    torch.cuda.synchronize()
    _, k, v64 = ref64.prepared(w, host)
    check_stored(w, host, ds.kv_prefill, k, v64)
    wd = gen.custom(f"b4d_{d}", 4, 2, d, [1] * n, [0] * n, seed=d, decode_from=0)
    hd = gen.make_inputs(wd, kv_dtype="e2m1", k_scale=KS, v_scale=VS)
    hd["qkv"] = host["qkv"]
    dd = run(wd, hd)
    _, k, v64 = ref64.prepared(wd, hd)
    check_stored(wd, hd, dd.kv_decode, k, v64)


def test_not_a_number_marks_its_block_and_infinity_is_clamped():
    from causal_gqa_attention_qkv_gb300 import attn, step
    w = gen.custom("nan4", 2, 1, 128, [3], [0], seed=3)
    host = gen.make_inputs(w, kv_dtype="e2m1", k_scale=KS, v_scale=VS)
    v = host["qkv"].view(3, 4, 128)[:, 3]
    v[0, 5] = float("nan")
    v[1, 40] = float("inf")
    v[2, 127] = float("-inf")
    ds = step.upload(w, host)
    attn.kv_append(ds.cfg, ds.qkv, ds.k_norm_w, ds.cu_seqlens, ds.kv_prefill, ds.workspace)
    kv = ds.kv_prefill
    e = ref64.entries(kv.v_cache, "e2m1", VS, kv.v_block_scale)[written_slots(host), 0]
    assert np.isnan(e[0, :16]).all() and np.isfinite(e[0, 16:]).all()
    assert e[1, 40] == 6 * 448 * VS and np.isfinite(e[1]).all()
    assert e[2, 127] == -6 * 448 * VS and np.isfinite(e[2]).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("d,ps", [(128, 0), (64, 64), (128, 128)])
def test_gather(kind, d, ps):
    """Entries of ranges of positions: whole requests, empty and partial ones."""
    from causal_gqa_attention_qkv_gb300 import attn, step
    lens = [300, 0, 65, 1]
    w = gen.custom(f"g_{kind}_{d}_{ps}", 6, 3, d, [1] * 4, lens, seed=d + ps, decode_from=0)
    host = gen.make_inputs(w, page_size=ps, kv_dtype=kind, k_scale=KS, v_scale=VS)
    ds = step.upload(w, host)
    kv = ds.kv_decode
    start, n = [7, 0, 0, 0], [293, 0, 65, 1]
    cu = torch.tensor([0] + np.cumsum(n).tolist(), dtype=torch.int32, device="cuda")
    k = torch.full((sum(n), 3, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, float("nan"))
    attn.kv_gather(ds.cfg, kv, cu, torch.tensor(start, dtype=torch.int32, device="cuda"), k, v, ds.workspace)
    torch.cuda.synchronize()
    assert ds.status() == 0
    slots = np.concatenate([ref64.slots_of(host, b, start[b] + n[b])[start[b]:] for b in range(4)])
    for got, cache, scale, bs in ((k, kv.k_cache, KS, kv.k_block_scale), (v, kv.v_cache, VS, kv.v_block_scale)):
        ref = ref64.entries(cache, kind, 1.0, bs)[slots].astype(np.float32)  # code (x block scale): exact
        ref = torch.from_numpy(ref * np.float32(scale if kind != "bf16" else 1)).bfloat16()
        assert torch.equal(got.cpu(), ref)


def test_gather_refuses_ranges_past_the_region():
    from causal_gqa_attention_qkv_gb300 import attn, step
    w = gen.custom("gr", 2, 1, 64, [1, 1], [70, 5], seed=1, decode_from=0)
    host = gen.make_inputs(w, page_size=64, kv_dtype="e2m1", k_scale=KS, v_scale=VS)
    ds = step.upload(w, host)
    out = [torch.full((6, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    call = lambda start, cu: attn.kv_gather(ds.cfg, ds.kv_decode, torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                            torch.tensor(start, dtype=torch.int32, device="cuda"), *out, ds.workspace)
    call([70, 0], [0, 3, 6])  # capacity 72: request 0 is skipped, request 1 is read
    assert ds.status() == attn.ATTN_STATUS_CAPACITY
    assert (out[0][:3] == 7).all() and (out[0][3:] != 7).any()
    call([0, -1], [0, 3, 6])
    assert ds.status() == attn.ATTN_STATUS_CAPACITY
    call([0, 0], [0, 3, 5])  # does not end at N
    assert ds.status() & attn.ATTN_STATUS_SEQLENS
    ds.kv_decode.page_table[0, 0] = -1
    call([0, 0], [0, 3, 6])
    assert ds.status() == attn.ATTN_STATUS_CAPACITY
    assert (out[0][:3] == 0).all()


def test_pages_outside_the_cache_read_as_bounded_entries():
    """A page number outside the pool: flagged, nothing faults, and the other
    request's rows stay right."""
    from causal_gqa_attention_qkv_gb300 import attn
    w = gen.custom("bad4", 8, 2, 128, [1, 1], [200, 300], seed=2, decode_from=0)
    host = gen.make_inputs(w, page_size=64, kv_dtype="e2m1", k_scale=KS, v_scale=VS)
    from causal_gqa_attention_qkv_gb300 import step
    ds = step.upload(w, host)
    ds.kv_decode.page_table[0, 1] = 1 << 20
    ds.run()
    assert ds.status() == attn.ATTN_STATUS_CAPACITY
    good = run(w, host)
    assert torch.equal(ds.out[1].view(torch.int16), good.out[1].view(torch.int16))


@pytest.mark.parametrize("hq,hkv,d,kind", [(8, 2, 128, "e2m1"), (8, 4, 64, "e2m1")])
def test_projected(hq, hkv, d, kind):
    """The fused projection stores the same format: V against its own fp32
    value (off by at most the accumulation's rounding, so up to a code at a
    boundary), then attention over what it stored."""
    from causal_gqa_attention_qkv_gb300 import attn, step
    lens, cache, C = [130, 1, 65], [0, 40, 200], 256
    w = gen.custom(f"proj4_{d}", hq, hkv, d, lens, cache, seed=d)
    host = gen.make_inputs(w, page_size=64, kv_dtype=kind, k_scale=KS, v_scale=VS)
    pj = gen.make_projection_inputs(w, hidden=C, seed=1)
    ds = step.upload(w, host)
    q = torch.empty(w.num_tokens, hq, d, dtype=torch.bfloat16, device="cuda")
    attn.qkv_proj_prepare(ds.cfg, pj["hidden"].cuda(), pj["w_qkv"].cuda(), ds.q_norm_w, ds.k_norm_w, ds.cu_seqlens,
                          ds.kv_prefill, q, ds.workspace)
    attn.prefill_attend(ds.cfg, q, ds.cu_seqlens, ds.max_seqlen, ds.kv_prefill, ds.out, ds.workspace)
    torch.cuda.synchronize()
    assert ds.status() == 0
    x = (pj["hidden"].double() @ pj["w_qkv"].double().T).numpy().reshape(-1, hq + 2 * hkv, d)
    at = ref64.places(host, d)
    q64 = ref64.norm_rope(x[:, :hq], host["q_norm_w"].double().numpy(), at, w.rms_eps, w.rope_theta)
    k64 = ref64.norm_rope(x[:, hq:hq + hkv], host["k_norm_w"].double().numpy(), at, w.rms_eps, w.rope_theta)
    slots, kv = written_slots(host), ds.kv_prefill
    for n, ref, scale in (("k", k64, KS), ("v", x[:, hq + hkv:], VS)):
        got = ref64.entries(getattr(kv, n + "_cache"), "e2m1", scale, getattr(kv, n + "_block_scale"))[slots]
        rc, rs = ref64.e2m1_store(ref, scale)
        want = (ref64.e2m1_value(rc).reshape(*rs.shape, 16) * ref64.e4m3_values()[rs][..., None]).reshape(ref.shape) * scale
        assert (got != want).mean() <= 2e-3
        # two code steps (a step is 2 s at most) where a boundary was crossed
        assert (np.abs(got - want) <= 3 * scale * np.repeat(ref64.e4m3_values()[np.minimum(rs + 1, 126)], 16, -1)).all()
    check_out(w, host, kv, ds.out, qkv=(q64, None, None))


def test_steps_replayed_from_a_graph():
    """A prefill and a decode call with a workspace each, captured and replayed:
    the eager bits."""
    from causal_gqa_attention_qkv_gb300 import step
    w = gen.custom("graph4", 16, 4, 128, [130, 1, 1], [0, 700, 5000], seed=9, decode_from=1)
    host = gen.make_inputs(w, page_size=64, kv_dtype="e2m1", k_scale=KS, v_scale=VS)
    a, b = run(w, host), step.upload(w, host)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run()
    for _ in range(3):
        b.out.fill_(float("nan"))
        g.replay()
    torch.cuda.synchronize()
    assert b.status() == 0
    assert torch.equal(a.out.view(torch.int16), b.out.view(torch.int16))
    for n in ("k_cache", "v_cache", "k_block_scale", "v_block_scale"):
        assert torch.equal(getattr(a.kv_decode, n), getattr(b.kv_decode, n)), n


def test_host_buffer_prefill_over_four_bits():
    from causal_gqa_attention_qkv_gb300 import step
    w = gen.custom("hp4", 8, 2, 128, [300, 40, 170], [10, 0, 64], seed=4)
    host = gen.make_inputs(w, page_size=64, kv_dtype="e2m1", k_scale=KS, v_scale=VS)
    a, b = run(w, host), step.upload(w, host)
    n = w.num_tokens
    q = torch.empty(n, 8, 128, dtype=torch.bfloat16, device="cuda")
    hp = step.HostPrefill(b.cfg, b.q_norm_w, b.k_norm_w, b.kv_prefill, b.workspace, b.qkv, q, b.out, chunk_tokens=128)
    out = torch.empty_like(b.out, device="cpu").pin_memory()
    hp.run(hp.plan(host["cu_seqlens"], host["cache_lens"]), host["qkv"].pin_memory(), out)
    torch.cuda.synchronize()
    assert hp.status() == 0
    for m in ("k_cache", "v_cache", "k_block_scale", "v_block_scale"):
        assert torch.equal(getattr(a.kv_prefill, m), getattr(b.kv_prefill, m)), m
    check_out(w, host, b.kv_prefill, out)


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (8, 1, 64), (3, 3, 64), (16, 2, 128)])
def test_a_cache_that_ends_with_its_last_request(hq, hkv, d):
    """No slot behind the last region, odd slot numbers, tiles that reach past the
    arrays: decode, prefill and gather give the bits of a cache with room behind it."""
    from causal_gqa_attention_qkv_gb300 import attn
    lens, new = [5, 71, 200], [1, 66, 3]
    g = torch.Generator().manual_seed(d + hq)
    cap = [c + n + 1 for c, n in zip(lens, new)]
    base = [0, cap[0], cap[0] + cap[1]]
    T = sum(cap)  # an odd start for the last two, nothing behind the last
    rand = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8)
    codes, blocks = rand(2, T, hkv, d // 2), torch.randint(0x28, 0x40, (2, hkv, T, d // 16), generator=g, dtype=torch.uint8)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cfg = attn.config(hq, hkv, d)
    W = (hq + 2 * hkv) * d
    qkv, one = [torch.randn(n, W, generator=g).bfloat16().cuda() for n in (sum(new), 3)]
    w = [(1 + 0.1 * torch.randn(d, generator=g)).bfloat16().cuda() for _ in range(2)]
    got = []
    for S in (T, T + 300):
        c = torch.full((2, S, hkv, d // 2), 0xFF, dtype=torch.uint8)
        b = torch.full((2, hkv, S, d // 16), 0x7F, dtype=torch.uint8)
        c[:, :T], b[:, :, :T] = codes, blocks
        c, b = c.cuda(), b.cuda()
        kv = attn.KVCache(c[0], c[1], torch.tensor(base, device="cuda"), i32(lens), i32(cap), None, 0, 0.04, 0.03, b[0].clone(),
                          b[1].clone())
        ws = attn.new_workspace(cfg, sum(new), 3, 512)
        out = torch.empty(sum(new), hq * d, dtype=torch.bfloat16, device="cuda")
        attn.prefill(cfg, qkv, w[0], w[1], i32([0, 1, 67, 70]), 66, kv, out, ws)
        kv.cache_lens += i32(new)
        dec = torch.empty(3, hq * d, dtype=torch.bfloat16, device="cuda")
        attn.decode(cfg, one, w[0], w[1], 203, kv, dec, ws)
        k, v = [torch.empty(T, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        attn.kv_gather(cfg, kv, i32([0, base[1], base[2], T]), i32([0, 0, 0]), k, v, ws)
        assert attn.get_status(ws) == 0
        got.append([x.view(torch.int16) for x in (out, dec, k, v)])
    for x, y in zip(*got):
        assert torch.equal(x, y)
    assert torch.isfinite(out).all() and torch.isfinite(dec).all()
