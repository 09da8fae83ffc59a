"""GPU tests of what calls read at their edges: pages whose number lies outside the
cache."""
import pytest
import torch

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
