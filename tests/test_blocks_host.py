"""CPU tests of the block calls and the calls on logits: the plain forms against
independent statements of the definitions, and every refusal that the host can see
(nothing is dereferenced or launched)."""
import ctypes

import numpy as np
import pytest
import torch

import ref_blocks as rb

FAKE = 1 << 20
PAST_CHECKS = (-4, -5)  # without a GPU a call that passes its checks stops at the device query


@pytest.fixture(scope="module")
def lib():
    from causal_gqa_attention_qkv_gb300 import attn, build
    build.build()
    return attn.load()


# ------------------------------------------------------------------ plain forms
def layout(cached, new, block=64, page=0):
    full = [c + n for c, n in zip(cached, new)]
    rows = [-(-n // block) for n in full]
    return {"block": block, "page": page, "cached": cached, "new": new, "table": None, "slots": sum(full) + 10,
            "base": [sum(full[:b]) for b in range(len(full))], "row_base": [sum(rows[:b]) for b in range(len(full))],
            "rows": sum(rows)}


def test_bounds_cover_full_blocks_only():
    c = layout([60, 0], [70, 63])
    keys = np.random.RandomState(0).randn(c["slots"], 2, 4)
    got = rb.bounds(c, keys)
    assert sorted(got) == [0, 1]  # 130 positions: blocks 0 (filled now) and 1; the second request fills none
    assert np.array_equal(got[1][1, 0], rb.bf16(keys[64:128, 1].min(0)))
    assert np.array_equal(got[0][0, 1], rb.bf16(keys[:64, 0].max(0)))
    assert sorted(rb.bounds(dict(c, cached=[64, 0], new=[66, 63]), keys)) == [1]
    assert sorted(rb.bounds(dict(c, cached=[64, 0], new=[66, 63]), keys, start=[-5, 0])) == [0, 1]


def test_score_is_the_sum_of_the_larger_products_and_bounds_every_key():
    rng = np.random.RandomState(1)
    q, keys = rng.randn(4, 16), rng.randn(3, 64, 16)
    lo, hi = keys.min(1), keys.max(1)
    s = rb.score(q, lo, hi)
    for i in range(3):
        assert np.isclose(s[i], np.maximum(q * lo[i], q * hi[i]).sum(), rtol=0, atol=1e-12)
        assert s[i] >= (keys[i] @ q.sum(0)).max() - 1e-12
    assert rb.score(q, np.full((1, 16), np.nan), hi[:1])[0] == np.inf


def test_select_takes_all_then_forced_then_best():
    c = layout([64 * 9 + 5], [1])
    q = np.ones((1, 1, 4))
    x = np.zeros((c["rows"], 1, 2, 4))
    x[:, 0, 1, 0] = [9, 1, 5, 5, 2, 5, 0, 8, 7, 99]
    assert rb.select(c, q, x, 1, 2, 12)[0, 0].tolist() == list(range(10)) + [-1, -1]
    assert rb.select(c, q, x, 1, 2, 5)[0, 0].tolist() == [0, 2, 7, 8, 9]  # 8, then the lowest of the fives
    assert rb.select(c, q, x, 0, 1, 4)[0, 0].tolist() == [0, 7, 8, 9]
    assert rb.select(c, q, x, 2, 2, 4)[0, 0].tolist() == [0, 1, 8, 9]


def test_attend_over_all_blocks_is_causal_attention():
    rng = np.random.RandomState(2)
    c = layout([100], [3])
    k, v, q = rng.randn(c["slots"], 1, 8), rng.randn(c["slots"], 1, 8), rng.randn(3, 2, 8)
    out, tol = rb.attend(c, q, np.tile(np.array([0, 1, -1], np.int32), (3, 1, 1)), k, v, False)
    for j in range(3):
        s = q[j] @ k[:101 + j, 0].T / np.sqrt(8)
        p = torch.softmax(torch.tensor(s), -1).numpy()
        assert np.allclose(out[j], p @ v[:101 + j, 0], rtol=0, atol=1e-12)
    assert (tol > 0).all()
    twice, _ = rb.attend(c, q, np.tile(np.array([1, 0, 1], np.int32), (3, 1, 1)), k, v, False)
    assert not np.allclose(out, twice)
    none, _ = rb.attend(c, q, np.full((3, 1, 2), -1, np.int32), k, v, False)
    assert (none == 0).all()


def test_adjust_follows_the_order_of_the_rules():
    x = np.array([2.0, -2.0, 1.0, 4.0, -np.inf], np.float32)
    seen = np.array([0, -32768, 3, -32767, 1], np.int16)
    y = rb.adjust(x, seen, rep=2.0, pres=0.5, freq=0.25, bias=[(0, 1.0), (3, 2.0), (0, 0.5), (9, 1.0)],
                  mask=np.array([True, True, True, True, True]))
    assert y.tolist() == [3.5, -4.0, 0.5 - 0.75 - 0.5, 3.0 - 0.25 - 0.5, -np.inf]
    assert rb.adjust(x, mask=np.zeros(5, bool)).tolist() == [-np.inf] * 5
    assert rb.adjust(x, seen, rep=-1.0).tolist() == x.tolist()


def test_seen_rows_count_and_stop():
    t = np.zeros((2, 8), np.int16)
    t[1, 3] = 0x7FFE
    got = rb.seen_rows(t, 5, [1, 0, 9], [[3, 3, 3, 7, -1], [2, 2], [1]])
    assert got[1, 3] == 0x7FFF and got[0, 2] == 2 and got[1, 7] == 0
    got = rb.seen_rows(got, 5, [0], [[2, 4]], prompt=True)
    assert got[0].tolist() == [0, 0, -32766, 0, -32768, 0, 0, 0]
    assert rb.seen_rows(got, 5, [0], [[1]], clear=True)[0].tolist() == [0, 1, 0, 0, 0, 0, 0, 0]


# ------------------------------------------------------------------ refusals
def make_kv(attn, **kw):
    f = dict(k_cache=FAKE, v_cache=FAKE, num_slots=1024, slot_base=None, cache_lens=FAKE, slot_capacity=FAKE,
             page_table=FAKE, page_size=128, pages_per_req=4, kv_dtype=0, k_scale=1.0, v_scale=1.0, k_block_scale=None,
             v_block_scale=None)
    return attn.AttnKV(*{**f, **kw}.values())


def make_blocks(attn, **kw):
    return attn.AttnBlocks(*{**dict(bounds=FAKE, num_rows=16, row_base=None, block_size=64), **kw}.values())


F = ctypes.c_void_p(FAKE)
ODD = ctypes.c_void_p(FAKE + 2)


def block_calls(lib, cfg=None, kv={}, blocks={}, no_kv=False, no_blocks=False, cu=F, B=2, N=3, q=F, lst=F, out=F, ws=F,
                nws=1 << 20, start=F, first=1, last=1, keep=4, max_kv=1000, bs=64):
    from causal_gqa_attention_qkv_gb300 import attn
    c = ctypes.byref(cfg or attn.config(8, 2, 64))
    k = None if no_kv else ctypes.byref(make_kv(attn, **kv))
    b = None if no_blocks else ctypes.byref(make_blocks(attn, **blocks))
    return dict(bounds=lib.attn_block_bounds(c, k, b, start, cu, B, ws, nws, None),
                select=lib.attn_block_select(c, q, cu, B, N, max_kv, k, b, first, last, keep, lst, ws, nws, None),
                attend=lib.attn_block_attend(c, q, cu, B, N, k, bs, lst, keep, out, ws, nws, None))


def refused(lib, names, code=-1, **kw):
    for name, rc in block_calls(lib, **kw).items():
        if name in names:
            assert rc == code, (name, kw, rc)
        else:
            assert rc in PAST_CHECKS, (name, kw, rc)


def test_row_numbers_have_32_bits(lib):
    refused(lib, set(), blocks={"num_rows": 2 ** 31 - 1})
    refused(lib, {"bounds", "select"}, blocks={"num_rows": 2 ** 31})
    refused(lib, {"bounds", "select"}, blocks={"num_rows": 2 ** 32 + 16})


def test_block_calls_check_their_arguments(lib):
    from causal_gqa_attention_qkv_gb300 import attn
    every = {"bounds", "select", "attend"}
    refused(lib, set())
    refused(lib, set(), N=0)
    refused(lib, set(), start=None)
    refused(lib, every, no_kv=True)
    refused(lib, {"bounds", "select"}, no_blocks=True)
    refused(lib, every, kv={"page_size": 48})
    refused(lib, every, code=-2, cfg=attn.config(8, 3, 64))
    for change in ({"bounds": None}, {"bounds": FAKE + 8}, {"num_rows": 0}, {"num_rows": 15}, {"block_size": 32},
                   {"block_size": 96}, {"block_size": 512}, {"block_size": 256}):  # 256 is more than a page
        refused(lib, {"bounds", "select"}, blocks=change)
    refused(lib, {"attend"}, bs=256)
    refused(lib, {"attend"}, bs=0)
    plain = {"page_table": None, "slot_base": FAKE}
    refused(lib, {"bounds", "select"}, kv=plain)  # contiguous: row_base is wanted
    refused(lib, set(), kv=plain, blocks={"row_base": FAKE, "num_rows": 1, "block_size": 256}, bs=256)
    refused(lib, {"bounds", "select"}, kv=plain, blocks={"row_base": FAKE + 4})
    refused(lib, every, B=-1)
    refused(lib, {"select", "attend"}, N=-1)
    refused(lib, {"select", "attend"}, cu=None)  # N != B
    refused(lib, set(), cu=None, N=2)
    refused(lib, every, cu=ODD)
    refused(lib, {"bounds"}, start=ODD)
    for bad in (None, ODD, ctypes.c_void_p(FAKE + 8)):
        refused(lib, {"select", "attend"}, q=bad)
        refused(lib, {"attend"}, out=bad)
    for bad in (None, ODD):
        refused(lib, {"select", "attend"}, lst=bad)
    refused(lib, {"select", "attend"}, keep=0)
    refused(lib, {"select", "attend"}, keep=4097)
    for change in ({"first": -1}, {"last": 0}, {"first": 4}, {"last": 5}, {"first": 2, "last": 3}, {"max_kv": 0},
                   {"max_kv": (1 << 24) + 1}, {"first": 2 ** 31 - 1, "last": 2}):
        refused(lib, {"select"}, **change)
    refused(lib, set(), first=3)
    refused(lib, every, code=-3, ws=None)
    refused(lib, every, code=-3, ws=ctypes.c_void_p(FAKE + 64))
    refused(lib, every, code=-3, nws=128)
    refused(lib, {"select"}, code=-3, nws=256)


def test_block_workspace_size(lib):
    from causal_gqa_attention_qkv_gb300 import attn
    cfg = attn.config(32, 8, 128)
    size = lambda *a: lib.attn_block_workspace_size(ctypes.byref(cfg), *a)
    assert size(1, 64, 64, 8) >= 256 + 8 * 12
    assert size(0, 64, 64, 8) == 256
    sizes = [size(n, 65536, 64, 64) for n in (1, 2, 64, 1000)]
    assert sizes == sorted(sizes) and sizes[2] >= 64 * 8 * 1024 * 12
    assert size(4, 1 << 24, 64, 4096) > size(4, 1 << 24, 128, 4096) > 0
    for bad in ((-1, 64, 64, 8), (1, 0, 64, 8), (1, (1 << 24) + 1, 64, 8), (1, 64, 32, 8), (1, 64, 64, 0), (1, 64, 64, 4097)):
        assert size(*bad) == 0
    assert lib.attn_block_workspace_size(ctypes.byref(attn.config(32, 5, 128)), 1, 64, 64, 8) == 0
    assert lib.attn_block_workspace_size(None, 1, 64, 64, 8) == 0


def test_logits_adjust_checks_its_arguments(lib):
    from causal_gqa_attention_qkv_gb300 import attn
    full = dict(seen=FAKE, seen_ld=1000, seen_rows=4, seen_row=FAKE, repetition=FAKE, presence=FAKE, frequency=FAKE,
                bias_start=FAKE, bias_token=FAKE, bias_value=FAKE, num_biases=9, mask=FAKE, mask_ld=32, mask_rows=2, mask_row=FAKE)

    def call(x=F, B=2, V=1000, ld=1000, out=ctypes.c_void_p(2 * FAKE), ldo=1000, no_rules=False, **kw):
        r = attn.AttnLogitsRules(*{**full, **kw}.values())
        return lib.attn_logits_adjust(x, B, V, ld, None if no_rules else ctypes.byref(r), out, ldo, None)
    ok = lambda **kw: call(**kw) in PAST_CHECKS
    assert ok() and ok(B=0) and ok(out=F) and ok(ld=1001) and ok(V=1)
    for name in ("seen", "seen_row", "repetition", "presence", "frequency", "mask", "mask_row", "bias_start"):
        assert ok(**{name: None}), name
    assert ok(num_biases=0, bias_token=None, bias_value=None) and ok(bias_start=None, num_biases=-1)
    assert ok(seen=None, seen_ld=0, seen_rows=0) and ok(mask=None, mask_ld=0, mask_rows=0)
    for kw in (dict(x=None), dict(out=None), dict(no_rules=True), dict(B=-1), dict(V=0), dict(V=(1 << 23) + 1, ld=1 << 24,
               ldo=1 << 24), dict(ld=999), dict(ldo=999), dict(out=F, ldo=1001), dict(x=ODD), dict(out=ODD),
               dict(seen=FAKE + 8), dict(seen_ld=992), dict(seen_ld=1001), dict(seen_rows=0), dict(bias_token=None),
               dict(bias_value=None), dict(num_biases=-1), dict(mask_ld=31), dict(mask_rows=0), dict(repetition=FAKE + 2), dict(mask=FAKE + 1),
               dict(seen_row=FAKE + 2), dict(bias_start=FAKE + 2), dict(mask_row=FAKE + 2)):
        assert call(**kw) == -1, kw


def test_tokens_seen_checks_its_arguments(lib):
    def call(seen=F, ld=1000, rows=4, V=1000, row=F, cu=F, tok=F, B=2, N=5, flags=0):
        return lib.attn_tokens_seen(seen, ld, rows, V, row, cu, tok, B, N, flags, None)
    ok = lambda **kw: call(**kw) in PAST_CHECKS
    assert ok() and ok(row=None) and ok(cu=None, N=2) and ok(flags=3) and ok(N=0, tok=None) and ok(B=0)
    for kw in (dict(seen=None), dict(seen=ctypes.c_void_p(FAKE + 8)), dict(ld=992), dict(ld=1001), dict(rows=0), dict(V=0),
               dict(V=1001), dict(row=ODD), dict(cu=ODD), dict(tok=ODD), dict(tok=None), dict(B=-1), dict(N=-1),
               dict(cu=None), dict(flags=4), dict(flags=-1), dict(V=(1 << 23) + 1, ld=1 << 24)):
        assert call(**kw) == -1, kw


def test_tokens_seen_takes_rows_of_any_length(lib):
    """What the grid of a call that empties rows cannot hold is refused, however large the product;
    the other calls do not touch whole rows."""
    def call(ld, B, flags):
        return lib.attn_tokens_seen(F, ld, 4, 1000, F, F, F, B, 5, flags, None)
    for ld, B in ((1 << 62, 1 << 15), ((1 << 63) - 8, 1), (1 << 45, 1), (1 << 23, 1 << 21), (8200, 1 << 30)):
        assert call(ld, B, 2) == call(ld, B, 3) == -1, (ld, B)
        assert call(ld, B, 0) in PAST_CHECKS and call(ld, B, 1) in PAST_CHECKS, (ld, B)
    for ld, B in ((1 << 43, 1), (1 << 32, 4000), (1 << 23, (1 << 21) - 1), (8192, 2 ** 31 - 1)):
        assert call(ld, B, 3) in PAST_CHECKS, (ld, B)
    assert call((1 << 44) - (1 << 13), 1, 3) in PAST_CHECKS and call(1 << 44, 1, 3) == -1
