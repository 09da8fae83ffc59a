"""GPU test that every call with a cfg and a cache refuses another model's cfg (the
refusal is the host's: nothing is launched)."""
import pytest
import torch

from test_gpu_pages import Pool, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_gqa_attention_qkv_gb300 import build
    build.build()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e2m1"])
def test_calls_refuse_another_models_cfg(kind):
    from causal_gqa_attention_qkv_gb300 import attn
    pool = Pool(kind, 8, 64, 2, 64, [70, 5], 2, 3)
    kv, one, st = pool.kv, i32([0]), pool.state()
    for h, d in ((4, 64), (2, 128)):  # twice the cache's bytes a slot
        cfg = attn.config(h, h, d)
        x, w = torch.zeros(2, 3 * h * d, dtype=torch.bfloat16, device="cuda"), torch.ones(d, dtype=torch.bfloat16, device="cuda")
        out, q = x[:, :h * d].contiguous(), torch.zeros(2, h, d, dtype=torch.bfloat16, device="cuda")
        cu, ws = i32([0, 1, 2]), attn.new_workspace(cfg, 2, 2, 192)
        wq = torch.zeros(3 * h * d, 64, dtype=torch.bfloat16, device="cuda")
        calls = (lambda: attn.pages_fork(cfg, kv, pool.ref, one, one, pool.ws),
                 lambda: attn.pages_copy(cfg, kv, one, one, pool.ws),
                 lambda: attn.pages_compact(cfg, kv, pool.ref, pool.ws),
                 lambda: attn.kv_gather(cfg, kv, cu, i32([0, 0]), q, q.clone(), ws),
                 lambda: attn.kv_append(cfg, x, w, cu, kv, ws),
                 lambda: attn.prefill(cfg, x, w, w, cu, 1, kv, out, ws),
                 lambda: attn.prefill_prepare(cfg, x, w, w, cu, kv, q, ws),
                 lambda: attn.prefill_attend(cfg, q, cu, 1, kv, out, ws),
                 lambda: attn.decode(cfg, x, w, w, 191, kv, out, ws),
                 lambda: attn.decode_attend(cfg, x, w, 191, kv, out, ws),
                 lambda: attn.decode_static_scratch(cfg, x, w, w, 191, kv, out),
                 lambda: attn.qkv_proj_prepare(cfg, x[:, :64].contiguous(), wq, w, w, cu, kv, q, ws))
        for call in calls:
            with pytest.raises(AssertionError, match="cfg"):
                call()
    with pytest.raises(AssertionError, match="cu_seqlens"):  # more requests than the table has rows
        cfg, q = attn.config(2, 2, 64), torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
        attn.kv_gather(cfg, kv, i32([0, 1, 2, 3]), i32([0, 0, 0]), q, q.clone(), pool.ws)
    assert pool.status() == 0
    for a, b in zip(pool.state(), st):
        assert torch.equal(a, b)
