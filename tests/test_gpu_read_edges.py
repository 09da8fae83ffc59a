"""GPU tests of what calls read at their edges: pages whose number lies outside the
cache, infinite entries under rotary axes, the precision of decode with axes."""
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


def bits(t):
    return t.view(torch.int16)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("hq,hkv,d,ps,lens,cache,bad", [
    (8, 2, 128, 64, [1, 1, 1], [200, 300, 5], 1),
    (16, 2, 64, 128, [1, 1, 1], [400, 900, 0], 2),            # groups of 8
    (4, 4, 128, 64, [1, 1, 1], [4000, 100, 64], 33),          # several splits
    (8, 2, 128, 64, [70, 3, 130], [200, 300, 0], 1),          # prefill, two pages per key tile
    (4, 2, 64, 64, [70, 3, 1], [200, 300, 0], 0),
    (8, 1, 64, 256, [70, 3, 130], [600, 300, 0], 1),
])
def test_a_page_outside_the_cache_reads_as_zeros(kind, hq, hkv, d, ps, lens, cache, bad):
    """The bits of the same call with a page of zeros in that place."""
    from causal_gqa_attention_qkv_gb300 import attn, step
    w = gen.custom(f"oob_{hq}_{d}_{ps}", hq, hkv, d, lens, cache, seed=d + ps, decode_from=0 if max(lens) == 1 else 3)
    host = gen.make_inputs(w, page_size=ps, kv_dtype=kind)
    free = sorted(set(range(host["k_cache"].shape[0] // ps)) - set(host["page_table"].flatten().tolist()))[0]
    for n in ("k_cache", "v_cache"):
        host[n][free * ps:free * ps + ps] = 0
    for n in ("k_block_scale", "v_block_scale"):
        if host[n] is not None:
            host[n][:, free * ps:free * ps + ps] = 0
    outs = []
    for page in (free, 1 << 20, -1, host["k_cache"].shape[0] // ps):
        ds = step.upload(w, host)
        (ds.kv_prefill or ds.kv_decode).page_table[0, bad] = page
        ds.run()
        assert ds.status() == (0 if page == free else attn.ATTN_STATUS_CAPACITY)
        outs.append(ds.out)
    assert torch.isfinite(outs[0]).all()
    for o in outs[1:]:
        assert torch.equal(bits(o), bits(outs[0]))


AXES = ([24, 20, 20], [12, 10, 10])


def axes_call(w, host, seed, top=5000):
    from causal_gqa_attention_qkv_gb300 import attn, step
    sections = AXES[0] if w.head_dim == 128 else AXES[1]
    pos = torch.randint(0, top, (3, w.batch), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
    ds = step.upload(w, host)
    return ds, pos, sections, attn.RopeAxes(pos.cuda(), sections, True)


def attend_within(w, host, q, keys, vals, h):
    """ref64.attend's derivation with Q and P rounded with half a step of h: (out, bound)."""
    cl, G, D = host["cache_lens"].numpy(), w.num_q_heads // w.num_kv_heads, w.head_dim
    out, tol = np.zeros_like(q), np.zeros_like(q)
    for b in range(w.batch):
        s = ref64.slots_of(host, b, int(cl[b]) + 1)
        for hd in range(w.num_q_heads):
            k, v, x = keys[s, hd // G], vals[s, hd // G], q[b, hd]
            sc = k @ x / np.sqrt(D)
            d = ((h + 2.0 ** -16) * np.abs(k) @ np.abs(x) + ref64.PAIR_REL * np.abs(k) @ ref64.pair_norm(x)) / np.sqrt(D)
            p = np.exp(sc - sc.max())
            p /= p.sum()
            out[b, hd] = p @ v
            grow = np.exp(2 * d.max()) - 1 + 2 * h + 2.0 ** -15
            tol[b, hd] = 2.0 ** -8 * 1.01 * np.abs(out[b, hd]) + grow * 1.01 * (p @ np.abs(v))
    return out, tol


@pytest.mark.parametrize("hq,hkv,d,cache,ps", [
    (32, 8, 128, [60, 700, 1, 3000], 0),
    (8, 1, 64, [9000, 300, 17], 64),              # groups of 8, several splits
    (3, 3, 128, [500, 5000], 0),
])
@pytest.mark.parametrize("attend", [False, True])
def test_decode_with_axes_keeps_q_and_p_to_sixteen_bits(attend, hq, hkv, d, cache, ps):
    """Norm weights of about 4 make the scores large, so that a Q rounded to bf16 alone
    moves the weights by several per cent of themselves: far outside this bound."""
    from causal_gqa_attention_qkv_gb300 import attn
    w = gen.custom(f"fineq_{hq}_{d}", hq, hkv, d, [1] * len(cache), cache, seed=d + hq, decode_from=0)
    host = gen.make_inputs(w, page_size=ps)
    host["q_norm_w"] = host["q_norm_w"] * 4
    ds, pos, sections, rope = axes_call(w, host, seed=d)
    kv = ds.kv_decode
    if attend:
        cu = torch.arange(w.batch + 1, dtype=torch.int32, device="cuda")
        attn.kv_append(ds.cfg, ds.qkv, ds.k_norm_w, cu, kv, ds.workspace, rope=rope)
        attn.decode_attend(ds.cfg, ds.qkv, ds.q_norm_w, ds.max_cache_len, kv, ds.out, ds.workspace, rope=rope)
    else:
        attn.decode(ds.cfg, ds.qkv, ds.q_norm_w, ds.k_norm_w, ds.max_cache_len, kv, ds.out, ds.workspace, rope=rope)
    assert ds.status() == 0
    q, _, _ = ref64.prepared(w, host, (pos.numpy(), sections, True))
    keys, vals = ref64.entries(kv.k_cache, "bf16", 1), ref64.entries(kv.v_cache, "bf16", 1)
    got = ds.out.double().cpu().numpy().reshape(q.shape)
    ref, tol = attend_within(w, host, q, keys, vals, 2.0 ** -16)
    assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) / tol).max())
    # the bound tells: with Q rounded to bf16 the oracle itself leaves it
    q16 = torch.from_numpy(q).bfloat16().double().numpy()
    plain, _ = attend_within(w, host, q16, keys, vals, 2.0 ** -16)
    assert (np.abs(plain - ref) > tol).any()


@pytest.mark.parametrize("d", [64, 128])
def test_decode_with_axes_where_the_values_cancel(d):
    """V such that the weighted sum is nearly 0: the output's own rounding is nothing
    there and a P rounded to bf16 alone leaves the bound."""
    from causal_gqa_attention_qkv_gb300 import attn
    h, cache = 4, [6 + b % 9 for b in range(24)]
    w = gen.custom(f"cancel_{d}", h, h, d, [1] * len(cache), cache, seed=d, decode_from=0)
    host = gen.make_inputs(w)
    host["qkv"].view(-1, 3 * h, d)[:, 2 * h:] = 0  # the new token's V
    ds, pos, sections, rope = axes_call(w, host, seed=d)
    q, k, _ = ref64.prepared(w, host, (pos.numpy(), sections, True))
    keys, vals = host["k_cache"].double().numpy(), host["v_cache"].double().numpy()
    keys[written_slots(host)] = torch.from_numpy(k).bfloat16().double().numpy()
    bf16 = lambda x: torch.from_numpy(x).bfloat16().double().numpy()
    rounded = np.zeros_like(q)
    for b, c in enumerate(cache):
        s = ref64.slots_of(host, b, c + 1)
        vals[s[c]] = 0
        for hd in range(h):
            p = np.exp(keys[s, hd] @ q[b, hd] / np.sqrt(d))
            p /= p.max()
            first, second = np.argsort(-p[:c])[:2]  # two heavy keys take the sum away, the second what the first left
            vals[s[first], hd] = vals[s[second], hd] = 0
            vals[s[first], hd] = -bf16(p @ vals[s, hd] / p[first])
            vals[s[second], hd] = -bf16(p @ vals[s, hd] / p[second])
            rounded[b, hd] = bf16(p) @ vals[s, hd] / p.sum()
    v = torch.from_numpy(vals).bfloat16()
    ds.v_cache[:v.shape[0]] = v.cuda()
    attn.decode(ds.cfg, ds.qkv, ds.q_norm_w, ds.k_norm_w, ds.max_cache_len, ds.kv_decode, ds.out, ds.workspace, rope=rope)
    assert ds.status() == 0
    keys = ref64.entries(ds.kv_decode.k_cache, "bf16", 1)
    ref, tol = attend_within(w, host, q, keys, vals, 2.0 ** -16)
    got = ds.out.double().cpu().numpy().reshape(q.shape)
    assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) / tol).max())
    assert (np.abs(rounded - ref) > tol).mean() > 0.1


@pytest.mark.parametrize("d", [64, 128])
def test_infinite_entries_under_axes(d):
    """An infinite V entry gives that infinity (every weight is positive here), an
    infinite K entry whose score is -inf takes no part: as in the call without axes."""
    from causal_gqa_attention_qkv_gb300 import attn, step
    w = gen.custom(f"inf_{d}", 4, 2, d, [1, 1, 1], [40, 300, 9], seed=d, decode_from=0)
    host = gen.make_inputs(w)
    slot = lambda b, p: int(host["slot_base"][b]) + p
    host["v_cache"][slot(0, 5), 0, 3] = float("inf")
    host["v_cache"][slot(1, 200), 1, 7] = float("-inf")
    host["k_cache"][slot(2, 4), 0, 0] = float("-inf")
    pos = torch.stack([torch.tensor([40, 300, 9], dtype=torch.int32)] * 3)  # the plain call's positions
    q, _, _ = ref64.prepared(w, host)
    heads = [h for h in (0, 1) if q[2, h, 0] > 0]  # of KV head 0: the score is -inf where q > 0
    assert heads
    plain, axes = step.upload(w, host), step.upload(w, host)
    plain.run()
    sections = AXES[0] if d == 128 else AXES[1]
    attn.decode(axes.cfg, axes.qkv, axes.q_norm_w, axes.k_norm_w, axes.max_cache_len, axes.kv_decode, axes.out,
                axes.workspace, rope=attn.RopeAxes(pos.cuda(), sections, True))
    assert plain.status() == 0 and axes.status() == 0
    a, b = plain.out.view(3, 4, d).float(), axes.out.view(3, 4, d).float()
    assert (a[0, :2, 3] == float("inf")).all() and (a[1, 2:, 7] == float("-inf")).all()
    assert (b[0, :2, 3] == float("inf")).all() and (b[1, 2:, 7] == float("-inf")).all()
    for h in heads:
        assert torch.isfinite(a[2, h]).all() and torch.isfinite(b[2, h]).all()
    assert torch.equal(torch.isfinite(a), torch.isfinite(b))


@pytest.mark.parametrize("hq,hkv,d,ps", [(8, 2, 128, 64), (6, 3, 64, 64), (8, 1, 64, 128), (16, 8, 64, 64)])
@pytest.mark.parametrize("extra", [1, 2, 3, 7])
def test_a_four_bit_pool_that_ends_inside_a_page(extra, hq, hkv, d, ps):
    """Heads' block scales then start at odd multiples of D / 16 bytes: the bits of a
    pool of whole pages, from decode, prefill and gather."""
    from causal_gqa_attention_qkv_gb300 import attn, step
    for lens, cache, df in (([1, 1, 1], [200, 3000, 5], 0), ([70, 3, 130], [200, 300, 0], 3)):
        w = gen.custom(f"tail_{hq}_{d}", hq, hkv, d, lens, cache, seed=d + hq, decode_from=df)
        host = gen.make_inputs(w, page_size=ps, kv_dtype="e2m1")
        more = dict(host)
        for n in ("k_cache", "v_cache"):
            more[n] = torch.cat([host[n], host[n][:extra]])
        for n in ("k_block_scale", "v_block_scale"):
            more[n] = torch.cat([host[n], host[n][:, :extra]], 1).contiguous()
        got = []
        for x in (host, more):
            ds = step.upload(w, x)
            ds.run()
            n = sum(cache)
            k, v = [torch.empty(n, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            cu = torch.tensor([0, cache[0], cache[0] + cache[1], n], dtype=torch.int32, device="cuda")
            attn.kv_gather(ds.cfg, ds.kv_prefill or ds.kv_decode, cu, torch.zeros(3, dtype=torch.int32, device="cuda"), k, v,
                           ds.workspace)
            assert ds.status() == 0
            got.append((ds.out, k, v))
        for a, b in zip(*got):
            assert torch.equal(bits(a), bits(b))
