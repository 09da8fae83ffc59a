"""CPU tests of the four-bit cache, the rotary axes and the page calls: the
64-bit references against independent statements of the definitions, and every
refusal that the host can see (nothing is dereferenced or launched)."""
import ctypes

import numpy as np
import pytest
import torch

import ref64

FAKE = 1 << 20
PAST_CHECKS = (-4, -5)  # without a GPU a call that passes its checks stops at the device query


@pytest.fixture(scope="module")
def lib():
    from causal_gqa_attention_qkv_gb300 import attn, build
    build.build()
    return attn.load()


# ------------------------------------------------------------------ references
def test_e4m3_values_are_torch_s():
    codes = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(ref64.e4m3_values(), codes.view(torch.float8_e4m3fn).double().numpy())


def test_e2m1_store_takes_the_nearest_representable_value():
    rng = np.random.RandomState(1)
    x = rng.randn(50, 3, 64).astype(np.float32)
    c, s = ref64.e2m1_store(x, 0.125)
    assert c.shape == x.shape and s.shape == (50, 3, 4)
    y = (x / 0.125).reshape(50, 3, 4, 16)
    sv = ref64.e4m3_values()[s][..., None]
    # the scale: no other E4M3 value is nearer to amax / 6
    target = np.abs(y).max(-1) / 6
    assert (np.abs(target[..., None] - ref64.e4m3_values()).min(-1) >= np.abs(target - sv[..., 0]) - 1e-12).all()
    grid = np.concatenate((-ref64.E2M1[::-1], ref64.E2M1))
    got = ref64.e2m1_value(c).reshape(y.shape)
    best = np.abs((y / sv)[..., None] - grid).min(-1)
    assert np.allclose(np.abs(y / sv - got), best, atol=1e-6)


def test_e2m1_ties_go_to_the_even_code():
    for mid, want in zip((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), (0, 1, 1, 2, 2, 4, 4)):
        x = np.zeros(16)
        x[0], x[1], x[2] = 6, mid, -mid
        c, s = ref64.e2m1_store(x, 1.0)
        assert ref64.e4m3_values()[s[0]] == 1
        assert ref64.e2m1_value(c)[1] == want and ref64.e2m1_value(c)[2] == -want


def test_inputs_draw_the_same_format():
    from causal_gqa_attention_qkv_gb300 import inputs as gen
    x = torch.randn(40, 2, 128, generator=torch.Generator().manual_seed(3)).bfloat16().float()
    codes, s = gen._e2m1_codes(x, 0.03125)
    c, rs = ref64.e2m1_store(x.numpy(), 0.03125)
    assert np.array_equal(s.numpy(), rs)
    assert np.array_equal(ref64.e2m1_value(ref64.unpack(codes)), ref64.e2m1_value(c))


def test_axis_order():
    assert ref64.axis_of(16, [4, 2, 2], False).tolist() == [0, 0, 0, 0, 1, 1, 2, 2]
    assert ref64.axis_of(16, [4, 2, 2], True).tolist() == [0, 1, 2, 0, 1, 2, 0, 0]
    a = ref64.axis_of(128, [24, 20, 20], True)
    assert [int((a == i).sum()) for i in range(3)] == [24, 20, 20]


def test_norm_rope_is_the_oracle_s():
    import oracle
    rng = np.random.RandomState(2)
    x, w = rng.randn(1, 1, 128), 1 + 0.1 * rng.randn(128)
    y = ref64.norm_rope(x, w, np.full((1, 64), 77.0), 1e-6, 1e6)
    assert np.allclose(y[0, 0], oracle.rope(oracle.rmsnorm(x[0, 0], w, 1e-6), 77, 1e6), rtol=0, atol=1e-12)


def test_attend_is_the_oracle_s():
    import oracle
    from causal_gqa_attention_qkv_gb300 import inputs as gen
    w = gen.custom("ref", 4, 2, 64, [5, 3], [7, 0], seed=1)
    host = gen.make_inputs(w)
    ref = oracle.step(oracle.cfg_of(w), host)
    q, _, _ = ref64.prepared(w, host)
    out, tol = ref64.attend(w, host, q, ref["k_cache"].double().numpy(), ref["v_cache"].double().numpy())
    assert np.allclose(out.reshape(-1, 64), ref["out"], rtol=0, atol=1e-9)
    assert (tol > 0).all()


# ------------------------------------------------------------------ refusals
def kv4(attn, **kw):
    f = dict(k_cache=FAKE, v_cache=FAKE, num_slots=1024, slot_base=FAKE, cache_lens=FAKE, slot_capacity=FAKE,
             page_table=None, page_size=0, pages_per_req=0, kv_dtype=2, k_scale=0.03, v_scale=0.06,
             k_block_scale=FAKE, v_block_scale=FAKE)
    return attn.AttnKV(*{**f, **kw}.values())


@pytest.mark.parametrize("change,ok", [
    ({}, True), ({"k_block_scale": None}, False), ({"v_block_scale": None}, False),
    ({"k_block_scale": FAKE + 8}, False), ({"v_block_scale": FAKE + 4}, False), ({"k_scale": 0.0}, False),
    ({"v_scale": float("inf")}, False), ({"k_scale": float("nan")}, False), ({"kv_dtype": 3}, False),
    ({"k_cache": FAKE + 8}, False)])
def test_four_bit_cache_checked_by_every_call(lib, change, ok):
    from causal_gqa_attention_qkv_gb300 import attn
    f, cfg = ctypes.c_void_p(FAKE), attn.config(32, 8, 128)
    c, k = ctypes.byref(cfg), ctypes.byref(kv4(attn, **change))
    n = 1 << 20
    for rc in (lib.attn_decode(c, f, f, f, 1, 4, k, f, f, n, None),
               lib.attn_decode_attend(c, f, f, 1, 4, k, f, f, n, None),
               lib.attn_decode_static_scratch(c, f, f, f, 1, 4, k, f, None, None),
               lib.attn_kv_append(c, f, f, f, f, 1, 4, k, f, n, None),
               lib.attn_prefill(c, f, f, f, f, 1, 4, 4, k, f, f, n, None),
               lib.attn_prefill_prepare(c, f, f, f, f, 1, 4, k, f, f, n, None),
               lib.attn_prefill_attend(c, f, f, 1, 4, 4, k, f, f, n, None),
               lib.attn_qkv_proj_prepare(c, f, 64, f, f, f, f, 1, 4, k, f, f, n, None),
               lib.attn_kv_gather(c, k, f, f, 1, 4, f, f, f, n, None)):
        assert (rc in PAST_CHECKS) if ok else rc == -1


def test_block_scales_are_read_for_four_bit_caches_only(lib):
    """A caller built against the struct without them ends at v_scale."""
    from causal_gqa_attention_qkv_gb300 import attn
    size = attn.AttnKV.k_block_scale.offset
    assert size == attn.AttnKV.v_scale.offset + 4 or size == attn.AttnKV.v_scale.offset + 8
    for dtype in (0, 1):
        kv = kv4(attn, kv_dtype=dtype, k_block_scale=None, v_block_scale=3)
        f = ctypes.c_void_p(FAKE)
        assert lib.attn_decode(ctypes.byref(attn.config(8, 2, 64)), f, f, f, 1, 4, ctypes.byref(kv), f, f, 1 << 20,
                               None) in PAST_CHECKS


def rope(attn, **kw):
    f = dict(num_axes=3, section=[24, 20, 20], interleaved=1, positions=FAKE, ld=8)
    f = {**f, **kw}
    sec = (ctypes.c_int32 * 4)(*(f["section"] + [0] * (4 - len(f["section"]))))
    return attn.AttnRopeAxes(f["num_axes"], sec, f["interleaved"], f["positions"], f["ld"])


@pytest.mark.parametrize("change,ok", [
    ({}, True), ({"interleaved": 0}, True), ({"ld": 4}, True), ({"ld": 3}, False), ({"ld": -1}, False),
    ({"positions": None}, False), ({"positions": FAKE + 2}, False), ({"num_axes": 0}, False), ({"num_axes": 5}, False),
    ({"section": [24, 20, 19]}, False), ({"section": [24, 20, 21]}, False), ({"section": [84, -10, -10]}, False),
    ({"section": [20, 22, 22]}, False), ({"section": [20, 22, 22], "interleaved": 0}, True),
    ({"num_axes": 1, "section": [64]}, True), ({"num_axes": 2, "section": [0, 64], "interleaved": 0}, True),
    ({"num_axes": 4, "section": [16, 16, 16, 16]}, True)])
def test_rope_axes_checked_by_every_call(lib, change, ok):
    from causal_gqa_attention_qkv_gb300 import attn
    f, cfg = ctypes.c_void_p(FAKE), attn.config(32, 8, 128)
    c, k, r = ctypes.byref(cfg), ctypes.byref(kv4(attn, kv_dtype=0)), ctypes.byref(rope(attn, **change))
    n = 1 << 20
    for rc in (lib.attn_kv_append_axes(c, f, f, f, 1, 4, k, r, f, n, None),
               lib.attn_prefill_prepare_axes(c, f, f, f, f, 1, 4, k, r, f, f, n, None),
               lib.attn_prefill_axes(c, f, f, f, f, 1, 4, 4, k, r, f, f, n, None),
               lib.attn_decode_axes(c, f, f, f, 4, 4, k, r, f, f, n, None),
               lib.attn_decode_attend_axes(c, f, f, 4, 4, k, r, f, f, n, None),
               lib.attn_qkv_proj_prepare_axes(c, f, 64, f, f, f, f, 1, 4, k, r, f, f, n, None)):
        assert (rc in PAST_CHECKS) if ok else rc == -1
    assert lib.attn_decode_axes(c, f, f, f, 4, 4, k, None, f, f, n, None) in PAST_CHECKS


def test_gather_arguments_checked(lib):
    from causal_gqa_attention_qkv_gb300 import attn
    f, odd, cfg = ctypes.c_void_p(FAKE), ctypes.c_void_p(FAKE + 8), attn.config(32, 8, 128)
    kv = kv4(attn)

    def call(cfg=cfg, kv=kv, cu=f, start=f, B=1, N=4, k=f, v=f, ws=f, n=256):
        return lib.attn_kv_gather(ctypes.byref(cfg), None if kv is None else ctypes.byref(kv), cu, start, B, N, k, v, ws,
                                  n, None)
    assert call() in PAST_CHECKS
    assert call(cfg=attn.config(32, 5, 128)) == -2
    for bad in ({"kv": None}, {"cu": None}, {"start": None}, {"B": -1}, {"N": -1}, {"k": None}, {"v": odd}, {"k": odd}):
        assert call(**bad) == -1, bad
    assert call(ws=None) == -3 and call(n=128) == -3


# ------------------------------------------------------------------ page calls
def paged(attn, **kw):
    return kv4(attn, **{**dict(num_slots=1000, slot_base=None, page_table=FAKE, page_size=64, pages_per_req=4), **kw})


def test_pages_workspace_size(lib):
    assert lib.attn_pages_workspace_size(1, 1) >= 256 + 5 * 4
    assert lib.attn_pages_workspace_size(1 << 24, 1 << 24) >= (3 + 2) * 4 << 24
    for pages, rows in ((0, 1), (1, 0), (-1, 5), ((1 << 24) + 1, 1), (1, (1 << 24) + 1)):
        assert lib.attn_pages_workspace_size(pages, rows) == 0


def test_page_calls_check_their_arguments(lib):
    from causal_gqa_attention_qkv_gb300 import attn
    f, cfg = ctypes.c_void_p(FAKE), attn.config(8, 2, 64)
    need = lib.attn_pages_workspace_size(15, 6)

    def calls(kv={}, pages={}, a=f, b=f, n=3, ws=f, nws=need, cfg=cfg, no_kv=False, no_pages=False):
        k = None if no_kv else ctypes.byref(paged(attn, **kv))
        p = None if no_pages else ctypes.byref(attn.AttnPages(*{**dict(page_table=FAKE, ref_count=FAKE, cache_lens=FAKE,
                                                                       num_rows=6), **pages}.values()))
        c = ctypes.byref(cfg)
        return dict(reserve=lib.attn_pages_reserve(k, p, a, b, n, ws, nws, None),
                    fork=lib.attn_pages_fork(c, k, p, a, b, n, ws, nws, None),
                    free=lib.attn_pages_free(k, p, a, n, ws, nws, None),
                    copy=lib.attn_pages_copy(c, k, a, b, n, ws, nws, None),
                    compact=lib.attn_pages_compact(c, k, p, ws, nws, None))

    every = {"reserve", "fork", "free", "copy", "compact"}

    def refused(names, code=-1, **kw):
        for name, rc in calls(**kw).items():
            if name in names:
                assert rc == code, (name, kw, rc)
            else:
                assert rc in PAST_CHECKS, (name, kw, rc)

    refused(set())
    refused(every, no_kv=True)
    refused(every - {"copy"}, no_pages=True)
    refused(every, kv={"page_table": None, "slot_base": FAKE})
    refused(every, kv={"page_size": 48})
    refused(every, kv={"num_slots": 63})                      # not one page
    refused(every, kv={"num_slots": (1 << 30) + 64}, nws=1 << 40)  # more than 2^24 pages
    refused(every, kv={"k_block_scale": None})
    for name in ("page_table", "ref_count", "cache_lens"):
        refused(every - {"copy"}, pages={name: None})
    refused(every - {"copy"}, pages={"num_rows": 0})
    refused({"reserve", "fork", "free", "copy"}, a=None)
    refused({"reserve", "fork", "copy"}, b=None)
    refused({"reserve", "fork", "free", "copy"}, n=-1)
    refused({"reserve", "fork"}, n=7)                         # more than the rows
    refused(every, code=-3, ws=None)
    refused(every, code=-3, ws=ctypes.c_void_p(FAKE + 64))
    refused({"reserve", "fork", "compact"}, code=-3, nws=need - 256)
    refused({"fork", "copy", "compact"}, code=-2, cfg=attn.config(8, 3, 64))
