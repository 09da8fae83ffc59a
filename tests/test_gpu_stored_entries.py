"""GPU tests of what the appends store over a four-bit cache, held to the format
where a code is decided: K to its exact value, far out in its positions too, V byte
for byte, and a K whose squares overflow."""
import dataclasses

import numpy as np
import pytest
import torch

import ref64
from causal_gqa_attention_qkv_gb300 import inputs as gen
from parity_util import written_slots

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_gqa_attention_qkv_gb300 import build
    build.build()


def stored(kv, name, slots):
    """(codes [n, Hkv, D], block scale codes [n, Hkv, D/16]) of some slots."""
    s = getattr(kv, f"{name}_block_scale")[:, torch.from_numpy(slots).cuda()].cpu().numpy().transpose(1, 0, 2)
    return ref64.unpack(getattr(kv, f"{name}_cache")[torch.from_numpy(slots).cuda()]), s.astype(np.int64)


# What one angle in fp32 pairs, absolute error 8e-8 below 2^24 positions, does to a
# rotated element, relative to its pair.
FINE_REL = 2.0 ** -23


def check_nearest(codes, scales, x, scale, off=None):
    """The codes and scales are those of a value that is off by err:
      err = 2^-24 |x| (x rounded to fp32) + off (FINE_REL pair), then the format's own
      fp32 roundings, 1 / scale, the product and the quotient: another 3 * 2^-24 |x|.
    A choice made for a value err away from x is at most 2 err further from x than
    the best choice."""
    y = (x / scale).reshape(*scales.shape, 16)
    off = FINE_REL * ref64.pair_norm(x) if off is None else off
    err = 2.0 ** -22 * np.abs(y) + (off / scale).reshape(y.shape)
    grid = ref64.e4m3_values()
    target = np.minimum(np.abs(y).max(-1) / 6, 448)
    best = np.abs(target[..., None] - grid).min(-1)
    assert (np.abs(target - grid[scales]) <= best + 2 * err.max(-1) / 6).all(), "block scales"
    sv = grid[scales][..., None]
    e = ref64.e2m1_value(codes).reshape(y.shape)
    best = np.full(y.shape, np.inf)
    for m in ref64.E2M1:
        best = np.minimum(best, np.abs(np.abs(y) - m * sv))
    far = (np.abs(e * sv - y) - best) / (2 * err)
    assert far.max() <= 1, f"{(far > 1).sum()} of {far.size} codes, {far.max():.1f} x the bound"


@pytest.mark.parametrize("d,theta,lo,hi", [
    (128, 1e6, 0, 1 << 16), (64, 1e6, 1 << 16, 1 << 20), (128, 1e6, 1 << 20, (1 << 24) + 1),
    (128, 1.05, 1 << 22, 1 << 23), (64, 1.05, 1 << 23, (1 << 24) + 1)])  # 1.05: every pair turns fast
@pytest.mark.parametrize("way", ["append", "decode"])
def test_k_is_coded_from_its_exact_value(way, d, theta, lo, hi):
    from causal_gqa_attention_qkv_gb300 import attn, step
    n, hkv = (6000, 2) if way == "append" else (1500, 4)
    lens = [n] if way == "append" else [1] * n
    w = gen.custom(f"kx_{d}", hkv, hkv, d, lens, [0] * len(lens), seed=d + hkv, decode_from=0 if way == "decode" else 1)
    w = dataclasses.replace(w, rope_theta=float(np.float32(theta)))  # the call's theta is an fp32 value
    host = gen.make_inputs(w, kv_dtype="e2m1", k_scale=0.03, v_scale=0.05)
    pos = torch.randint(lo, hi, (1, n), generator=torch.Generator().manual_seed(d), dtype=torch.int32)
    pos[0, -1] = hi - 1
    ds = step.upload(w, host)
    rope = attn.RopeAxes(pos.cuda(), [d // 2])
    if way == "append":
        attn.kv_append(ds.cfg, ds.qkv, ds.k_norm_w, ds.cu_seqlens, ds.kv_prefill, ds.workspace, rope=rope)
    else:
        attn.decode(ds.cfg, ds.qkv, ds.q_norm_w, ds.k_norm_w, 0, ds.kv_decode, ds.out, ds.workspace, rope=rope)
    assert ds.status() == 0
    _, k, _ = ref64.prepared(w, host, (pos.numpy(), [d // 2], False))
    check_nearest(*stored(ds.kv_prefill or ds.kv_decode, "k", written_slots(host)), k, host["k_scale"])


def test_k_far_out_in_a_paged_cache():
    """The positions of the cache itself, just below 2^24: the last page of the row."""
    from causal_gqa_attention_qkv_gb300 import attn
    d, n, ps = 64, 4000, 1 << 20
    w = dataclasses.replace(gen.custom("kfar", 1, 1, d, [n], [(1 << 24) - n], seed=3), rope_theta=float(np.float32(1.05)))
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn(n, 3 * d, generator=g).bfloat16()
    kw = (1 + 0.1 * torch.randn(d, generator=g)).bfloat16()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    code = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")
    kv = attn.KVCache(code(ps, 1, d // 2), code(ps, 1, d // 2), torch.zeros(1, dtype=torch.int64, device="cuda"),
                      i32([(1 << 24) - n]), i32([1 << 24]), i32([[-1] * 15 + [0]]), ps, 0.03, 0.05, code(1, ps, d // 16),
                      code(1, ps, d // 16))
    cfg = attn.config(1, 1, d, w.rms_eps, w.rope_theta)
    ws = attn.new_workspace(cfg, n, 1, 256)
    attn.kv_append(cfg, qkv.cuda(), kw.cuda(), i32([0, n]), kv, ws)
    assert attn.get_status(ws) == 0
    place = np.repeat(np.arange((1 << 24) - n, 1 << 24)[:, None], d // 2, 1).astype(np.float64)
    k = ref64.norm_rope(qkv.view(n, 3, d)[:, 1:2].double().numpy(), kw.double().numpy(), place, w.rms_eps, w.rope_theta)
    check_nearest(*stored(kv, "k", np.arange(ps - n, ps)), k, 0.03)


@pytest.mark.parametrize("d", [64, 128])
def test_k_of_many_tokens_near_the_last_position(d):
    """Enough elements that an angle off by some 1e-5 now and then shows: fp32 quotients
    by pi / 2 are off by one there.  The definition in fp64 on the device."""
    from causal_gqa_attention_qkv_gb300 import attn
    n, hkv, scale = 200000, 2, 0.03
    theta = float(np.float32(1.05))
    g = torch.Generator(device="cuda").manual_seed(d)
    qkv = torch.randn(n, 3 * hkv * d, generator=g, device="cuda").bfloat16()
    kw = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).bfloat16()
    pos = torch.randint(13 << 20, (1 << 24) + 1, (1, n), generator=g, device="cuda", dtype=torch.int32)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    code = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")
    kv = attn.KVCache(code(n, hkv, d // 2), code(n, hkv, d // 2), torch.zeros(1, dtype=torch.int64, device="cuda"), i32([0]),
                      i32([n]), None, 0, scale, 0.05, code(hkv, n, d // 16), code(hkv, n, d // 16))
    cfg = attn.config(hkv, hkv, d, 1e-6, theta)
    ws = attn.new_workspace(cfg, 1, 1, 256)
    attn.kv_append(cfg, qkv, kw, i32([0, n]), kv, ws, rope=attn.RopeAxes(pos, [d // 2]))
    assert attn.get_status(ws) == 0
    grid = torch.from_numpy(ref64.e4m3_values()).cuda()
    freq = theta ** (-2.0 * torch.arange(d // 2, device="cuda", dtype=torch.float64) / d)
    for t in range(0, n, 20000):
        x = qkv[t:t + 20000].double().view(-1, 3 * hkv, d)[:, hkv:2 * hkv]
        x = x * kw.double() / (x.square().mean(-1, keepdim=True) + cfg.rms_eps).sqrt()
        a = (pos[0, t:t + 20000].double()[:, None] * freq)[:, None]
        c, s = x.chunk(2, -1)
        y = torch.cat((c * a.cos() - s * a.sin(), s * a.cos() + c * a.sin()), -1) / scale
        pair = torch.hypot(y, y.roll(d // 2, -1))
        err = (2.0 ** -22 * y.abs() + FINE_REL * pair).unflatten(-1, (-1, 16))  # as in check_nearest
        y = y.unflatten(-1, (-1, 16))
        sv = grid[kv.k_block_scale[:, t:t + 20000].transpose(0, 1).long()][..., None]
        b = kv.k_cache[t:t + 20000].long()
        m = torch.from_numpy(ref64.E2M1).cuda()
        e = m[torch.stack((b & 7, b >> 4 & 7), -1).flatten(-2)].unflatten(-1, (-1, 16))
        sign = torch.stack((b & 8, b >> 4 & 8), -1).flatten(-2).unflatten(-1, (-1, 16)) != 0
        off = (torch.where(sign, -e, e) * sv - y).abs()
        best = torch.stack([(y.abs() - v * sv).abs() for v in m.tolist()]).amin(0)
        assert (off <= best + 2 * err).all(), float(((off - best) / err).max())
        target = y.abs().amax(-1) / 6
        near = torch.searchsorted(grid, target).clamp(1, len(grid) - 1)
        best = torch.minimum((target - grid[near]).abs(), (target - grid[near - 1]).abs())
        assert ((target - sv[..., 0]).abs() <= best + 2 * err.amax(-1) / 6).all()


def signed_zeros_and_borders(d, scale):
    """bf16 rows [n, 2, D]: +0 and -0 among other entries, blocks of -0 alone, tiny
    negative entries beside large ones, ordinary values, values next to borders."""
    rng = np.random.RandomState(d)
    x = rng.randn(64, 2, d)
    x[rng.rand(*x.shape) < 0.2] = -0.0
    x[rng.rand(*x.shape) < 0.1] = 0.0
    x[3, 0] = -0.0
    x[4, 1, :d // 2] *= -1e-30
    x[5] = -np.abs(x[5]) * 1e-3
    x[5, :, ::16] = 7
    x[6:40] = rng.choice([0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6], (34, 2, d)) * rng.choice([-1, 1], (34, 2, d)) * scale
    return torch.from_numpy(x.astype(np.float32)).bfloat16()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [0.0625, 0.0371, 1.7, 1e-4])
def test_v_bytes_are_the_formats(d, scale):
    """V's bytes, signs of zeros among them, for scales that are no powers of two
    too (the product with the rounded reciprocal is inexact there)."""
    from causal_gqa_attention_qkv_gb300 import attn, step
    v = signed_zeros_and_borders(d, scale)
    n = v.shape[0]
    for lens, df in (([n], 1), ([1] * n, 0)):
        w = gen.custom(f"vb_{d}", 4, 2, d, lens, [0] * len(lens), seed=d, decode_from=df)
        host = gen.make_inputs(w, kv_dtype="e2m1", k_scale=0.03, v_scale=scale)
        host["qkv"].view(n, 8, d)[:, 6:] = v
        ds = step.upload(w, host)
        ds.run()
        assert ds.status() == 0
        codes, scales = stored(ds.kv_prefill or ds.kv_decode, "v", written_slots(host))
        want, blocks = ref64.e2m1_store(v.float().numpy(), scale)
        assert np.array_equal(scales, blocks)
        assert np.array_equal(codes, want), f"{(codes != want).mean():.2%}"


@pytest.mark.parametrize("d", [64, 128])
def test_k_whose_squares_overflow_is_stored_as_over_a_bf16_cache(d):
    """Arithmetic is fp32: a mean of squares past its range makes the normed head 0,
    whatever the cache holds, and marks nothing as no number."""
    from causal_gqa_attention_qkv_gb300 import attn, step
    for lens, df in (([5], 1), ([1] * 5, 0)):
        w = gen.custom(f"ov_{d}", 4, 2, d, lens, [0] * len(lens), seed=d, decode_from=df)
        got = []
        for kind in ("bf16", "e2m1"):
            host = gen.make_inputs(w, kv_dtype=kind, k_scale=0.03, v_scale=0.05)
            host["qkv"].view(5, 8, d)[2, 4, 7] = 1e25
            ds = step.upload(w, host)
            cu = torch.tensor([0] + np.cumsum(lens).tolist(), dtype=torch.int32, device="cuda")
            kv = ds.kv_prefill or ds.kv_decode
            if df:
                attn.kv_append(ds.cfg, ds.qkv, ds.k_norm_w, cu, kv, ds.workspace)
            else:
                ds.run()
            assert ds.status() == 0
            got.append(ref64.entries(kv.k_cache, kind, 0.03 if kind == "e2m1" else 1, kv.k_block_scale)[written_slots(host)])
        assert (got[0][2, 0] == 0).all() and (got[1][2, 0] == 0).all()
        assert np.isfinite(got[1]).all() and (got[1][2, 1] != 0).any() and (got[1][1, 0] != 0).any()
