"""GPU tests of rotary positions with several axes: the prologue, decode and the
fused projection against the 64-bit definition, for every order of axes and
every cache type; equal positions on all axes give the plain call's bits."""
import numpy as np
import pytest
import torch

import ref64
from causal_gqa_attention_qkv_gb300 import inputs as gen
from parity_util import bf16_step, written_slots

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_gqa_attention_qkv_gb300 import build
    build.build()


def positions(axes, n, seed, top=100000):
    return torch.randint(0, top, (axes, n), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)


def within_half_step(got, ref, step_rel):
    """|got - ref| within half a step of a float type (relative step_rel / 2 of
    either side) plus the fp32 error of the element's rotation pair."""
    err = np.abs(got - ref)
    tol = step_rel * np.maximum(np.abs(got), np.abs(ref)) + ref64.PAIR_REL * ref64.pair_norm(ref) + 2.0 ** -25
    assert (err <= tol).all(), float((err / tol).max())


CASES = [
    # (Hq, Hkv, D, new lens, cached lens, sections, interleaved, cache, page size)
    (32, 8, 128, [300, 1, 77], [0, 5, 200], [24, 20, 20], True, "bf16", 0),
    (16, 2, 128, [130, 65], [0, 7], [16, 24, 24], False, "bf16", 64),
    (8, 8, 64, [33, 257], [3, 0], [12, 10, 10], True, "e4m3", 0),
    (6, 3, 128, [257, 31], [0, 100], [0, 32, 32], False, "e2m1", 64),
    (4, 2, 64, [1], [0], [8, 8, 8, 8], False, "bf16", 0),
    (4, 1, 64, [9, 2], [0, 64], [32], True, "bf16", 0),
    (16, 4, 128, [64, 2], [1, 0], [34, 30], True, "e2m1", 0),
]


def make(case, decode=False):
    hq, hkv, d, lens, cache, sections, inter, kind, ps = case
    if decode:
        lens = [1] * len(cache)
    w = gen.custom(f"ax_{hq}_{hkv}_{d}_{kind}_{inter}", hq, hkv, d, lens, cache, seed=hq + d + len(sections),
                   decode_from=0 if decode else len(lens))
    return w, gen.make_inputs(w, page_size=ps, kv_dtype=kind)


@pytest.mark.parametrize("case", CASES)
def test_prepare_then_attend(case):
    from causal_gqa_attention_qkv_gb300 import attn, step
    hq, hkv, d, _, _, sections, inter, kind, _ = case
    w, host = make(case)
    n = w.num_tokens
    pos = positions(len(sections), n + 3, seed=d)[:, 1:n + 1]  # rows longer than N: a strided view
    ds = step.upload(w, host)
    wide = torch.zeros(len(sections), n + 3, dtype=torch.int32, device="cuda")
    wide[:, 1:n + 1] = pos.cuda()
    rope = attn.RopeAxes(wide[:, 1:n + 1], sections, inter)
    q = torch.empty(n, hq, d, dtype=torch.bfloat16 if kind == "bf16" else torch.float16, device="cuda")
    attn.prefill_prepare(ds.cfg, ds.qkv, ds.q_norm_w, ds.k_norm_w, ds.cu_seqlens, ds.kv_prefill,
                         q.view(torch.bfloat16), ds.workspace, rope=rope)
    attn.prefill_attend(ds.cfg, q.view(torch.bfloat16), ds.cu_seqlens, ds.max_seqlen, ds.kv_prefill, ds.out, ds.workspace)
    torch.cuda.synchronize()
    assert ds.status() == 0
    q64, k64, _ = ref64.prepared(w, host, (pos.numpy(), sections, inter))
    half = 2.0 ** -8 if kind == "bf16" else 2.0 ** -11
    within_half_step(q.double().cpu().numpy(), q64, half)
    kv, slots = ds.kv_prefill, written_slots(host)
    keys = ref64.entries(kv.k_cache, kind, host["k_scale"] if kind != "bf16" else 1, kv.k_block_scale)
    vals = ref64.entries(kv.v_cache, kind, host["v_scale"] if kind != "bf16" else 1, kv.v_block_scale)
    if kind == "bf16":
        within_half_step(keys[slots], k64, half)
    ref, tol = ref64.attend(w, host, q64, keys, vals)
    assert (np.abs(ds.out.double().cpu().numpy().reshape(ref.shape) - ref) <= tol).all()
    # the one call, and the K/V append alone, give the same bits
    e = step.upload(w, host)
    attn.prefill(e.cfg, e.qkv, e.q_norm_w, e.k_norm_w, e.cu_seqlens, e.max_seqlen, e.kv_prefill, e.out, e.workspace,
                 rope=rope)
    f = step.upload(w, host)
    attn.kv_append(f.cfg, f.qkv, f.k_norm_w, f.cu_seqlens, f.kv_prefill, f.workspace, rope=rope)
    torch.cuda.synchronize()
    assert torch.equal(e.out.view(torch.int16), ds.out.view(torch.int16))
    for x in (e, f):
        assert torch.equal(x.k_cache.view(torch.uint8), ds.k_cache.view(torch.uint8))
        assert torch.equal(x.v_cache.view(torch.uint8), ds.v_cache.view(torch.uint8))


@pytest.mark.parametrize("case", CASES)
def test_decode(case):
    from causal_gqa_attention_qkv_gb300 import attn, step
    hq, hkv, d, _, cache, sections, inter, kind, _ = case
    w, host = make(case, decode=True)
    pos = positions(len(sections), w.batch, seed=d + 1)
    rope = attn.RopeAxes(pos.cuda(), sections, inter)
    a, b = step.upload(w, host), step.upload(w, host)
    attn.decode(a.cfg, a.qkv, a.q_norm_w, a.k_norm_w, a.max_cache_len, a.kv_decode, a.out, a.workspace, rope=rope)
    cu = torch.arange(w.batch + 1, dtype=torch.int32, device="cuda")
    attn.kv_append(b.cfg, b.qkv, b.k_norm_w, cu, b.kv_decode, b.workspace, rope=rope)
    attn.decode_attend(b.cfg, b.qkv, b.q_norm_w, b.max_cache_len, b.kv_decode, b.out, b.workspace, rope=rope)
    torch.cuda.synchronize()
    assert a.status() == 0 and b.status() == 0
    assert torch.equal(a.out.view(torch.int16), b.out.view(torch.int16))
    assert torch.equal(a.k_cache.view(torch.uint8), b.k_cache.view(torch.uint8))
    kv = a.kv_decode
    q64, k64, _ = ref64.prepared(w, host, (pos.numpy(), sections, inter))
    keys = ref64.entries(kv.k_cache, kind, host["k_scale"] if kind != "bf16" else 1, kv.k_block_scale)
    vals = ref64.entries(kv.v_cache, kind, host["v_scale"] if kind != "bf16" else 1, kv.v_block_scale)
    if kind == "bf16":
        within_half_step(keys[written_slots(host)], k64, 2.0 ** -8)
    ref, tol = ref64.attend(w, host, q64, keys, vals)
    assert (np.abs(a.out.double().cpu().numpy().reshape(ref.shape) - ref) <= tol).all()


@pytest.mark.parametrize("kind", ["bf16", "e2m1"])
@pytest.mark.parametrize("d", [64, 128])
def test_same_position_on_every_axis_is_the_plain_call(d, kind):
    from causal_gqa_attention_qkv_gb300 import attn, step
    lens, cache = [70, 1, 130], [0, 300, 5]
    w = gen.custom(f"axeq_{d}_{kind}", 8, 2, d, lens, cache, seed=d)
    host = gen.make_inputs(w, kv_dtype=kind)
    p = torch.cat([torch.arange(c, c + n) for c, n in zip(cache, lens)]).int()
    rope = attn.RopeAxes(p.repeat(3, 1).cuda(), [d // 2 - 20, 10, 10], True)
    a, b = step.upload(w, host), step.upload(w, host)
    a.run()
    attn.prefill(b.cfg, b.qkv, b.q_norm_w, b.k_norm_w, b.cu_seqlens, b.max_seqlen, b.kv_prefill, b.out, b.workspace,
                 rope=rope)
    torch.cuda.synchronize()
    assert torch.equal(a.out.view(torch.int16), b.out.view(torch.int16))
    assert torch.equal(a.k_cache.view(torch.uint8), b.k_cache.view(torch.uint8))


@pytest.mark.parametrize("d,kind", [(128, "bf16"), (64, "e4m3"), (128, "e2m1")])
def test_projected(d, kind):
    from causal_gqa_attention_qkv_gb300 import attn, step
    hq, hkv, lens, cache, C = 8, 2, [130, 1, 65], [0, 40, 200], 256
    w = gen.custom(f"axproj_{d}_{kind}", hq, hkv, d, lens, cache, seed=d)
    host = gen.make_inputs(w, kv_dtype=kind)
    pj = gen.make_projection_inputs(w, hidden=C, seed=2)
    sections, n = [d // 2 - 20, 10, 10], w.num_tokens
    pos = positions(3, n, seed=7)
    ds = step.upload(w, host)
    q = torch.empty(n, hq, d, dtype=torch.bfloat16 if kind == "bf16" else torch.float16, device="cuda")
    attn.qkv_proj_prepare(ds.cfg, pj["hidden"].cuda(), pj["w_qkv"].cuda(), ds.q_norm_w, ds.k_norm_w, ds.cu_seqlens,
                          ds.kv_prefill, q, ds.workspace, rope=attn.RopeAxes(pos.cuda(), sections, True))
    torch.cuda.synchronize()
    assert ds.status() == 0
    x = (pj["hidden"].double() @ pj["w_qkv"].double().T).numpy().reshape(n, hq + 2 * hkv, d)
    at = ref64.places(host, d, (pos.numpy(), sections, True))
    q64 = ref64.norm_rope(x[:, :hq], host["q_norm_w"].double().numpy(), at, w.rms_eps, w.rope_theta)
    # the fp32 accumulation of 256 products is off by at most 256 * 2^-24 of
    # their magnitudes' sum, here taken relative to the head's largest value
    got = q.double().cpu().numpy()
    half = 2.0 ** -8 if kind == "bf16" else 2.0 ** -11
    mag = (pj["hidden"].double().abs() @ pj["w_qkv"].double().abs().T).numpy().reshape(n, hq + 2 * hkv, d)[:, :hq]
    rms = np.sqrt((x[:, :hq] ** 2).mean(-1, keepdims=True))
    acc = 1.5 * C * 2.0 ** -24 * mag.max(-1, keepdims=True) / rms * 4
    assert (np.abs(got - q64) <= half * np.maximum(np.abs(got), np.abs(q64)) + ref64.PAIR_REL * ref64.pair_norm(q64) + acc).all()


def test_positions_out_of_range_skip_the_token():
    from causal_gqa_attention_qkv_gb300 import attn, step
    w = gen.custom("axbad", 8, 2, 128, [6], [0], seed=5)
    host = gen.make_inputs(w)
    for value in (-1, (1 << 24) + 1):
        pos = positions(3, 6, seed=1)
        pos[1, 2] = value
        ds = step.upload(w, host)
        q = torch.full((6, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        rope = attn.RopeAxes(pos.cuda(), [24, 20, 20], True)
        attn.prefill_prepare(ds.cfg, ds.qkv, ds.q_norm_w, ds.k_norm_w, ds.cu_seqlens, ds.kv_prefill, q, ds.workspace,
                             rope=rope)
        assert ds.status() == attn.ATTN_STATUS_POSITION
        s = written_slots(host)
        same = (ds.k_cache.cpu().view(torch.int16) == host["k_cache"].view(torch.int16)).flatten(1).all(1)[s]
        assert same.tolist() == [False, False, True, False, False, False]
        assert (q[2] == 7).all() and not (q[1] == 7).any() and not (q[3] == 7).all()
    pos = positions(3, 2, seed=1)
    pos[2, 1] = -5
    wd = gen.custom("axbadd", 8, 2, 128, [1, 1], [30, 700], seed=6, decode_from=0)
    ds = step.upload(wd, gen.make_inputs(wd))
    ds.out.fill_(7)
    attn.decode(ds.cfg, ds.qkv, ds.q_norm_w, ds.k_norm_w, ds.max_cache_len, ds.kv_decode, ds.out, ds.workspace,
                rope=attn.RopeAxes(pos.cuda(), [24, 20, 20], False))
    assert ds.status() == attn.ATTN_STATUS_POSITION
    assert (ds.out[1] == 7).all() and (ds.out[0] != 7).any()


@pytest.mark.parametrize("kind,ps", [("bf16", 0), ("e4m3", 64), ("e2m1", 64)])
def test_decode_of_a_batch_whose_heads_fill_the_card(kind, ps):
    """Splits of 2048 keys (B Hkv = 320): requests of one split beside some of three."""
    cache = [int(x) for x in np.linspace(0, 2100, 38)] + [4500, 2047]
    test_decode((16, 8, 64, [], cache, [12, 10, 10], True, kind, ps))
