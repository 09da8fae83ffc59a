"""GPU test that a step's count of launches is what it launches: partial results are
written to the workspace exactly where a merge is counted."""
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


@pytest.mark.parametrize("kind,B,top,launches", [
    ("bf16", 64, 2000, 2), ("e4m3", 64, 2000, 2), ("e2m1", 64, 2000, 1), ("e2m1", 64, 5000, 2), ("e2m1", 2, 200, 1),
    ("e2m1", 2, 700, 2), ("bf16", 2, 200, 1)])
def test_launches_of_a_decode_step(kind, B, top, launches):
    from causal_gqa_attention_qkv_gb300 import step
    lens = [max(0, top - 1 - 17 * b) for b in range(B)]
    w = gen.custom(f"launch_{kind}_{B}", 16, 8, 64, [1] * B, lens, seed=B, decode_from=0)
    ds = step.upload(w, gen.make_inputs(w, kv_dtype=kind))
    ds.workspace[256:] = 0xA5
    ds.run()
    assert ds.status() == 0
    assert ds.launches() == launches
    assert bool((ds.workspace[256:] != 0xA5).any()) == (launches == 2)
