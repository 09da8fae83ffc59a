"""GPU tests of what calls read at their edges: pages whose number lies outside the
cache, infinite entries under rotary axes."""
import pytest
import torch

import ref64
from causal_gqa_attention_qkv_gb300 import inputs as gen

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
