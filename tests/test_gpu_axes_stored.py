"""GPU tests of the entries that the calls with rotary axes store, K and V, for
every cache type: each is the nearest of its type to the 64-bit definition, up to
the error of the value that was rounded."""
import numpy as np
import pytest
import torch

import ref64
from causal_gqa_attention_qkv_gb300 import inputs as gen
from parity_util import written_slots
from test_gpu_axes import CASES, make, positions
from test_gpu_stored_entries import check_nearest, stored

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_gqa_attention_qkv_gb300 import build
    build.build()


def check_entries(kind, kv, host, name, x, off):
    """Entries of the written slots against x [n, Hkv, D], computed to within off."""
    slots, scale = written_slots(host), host[f"{name}_scale"]
    if kind == "e2m1":
        return check_nearest(*stored(kv, name, slots), x, scale, off)
    got = ref64.entries(getattr(kv, f"{name}_cache"), kind, 1.0)[slots]
    if kind == "bf16":
        # half a step of either side's binade
        tol = 2.0 ** -8 * np.maximum(np.abs(got), np.abs(x)) + off
        assert (np.abs(got - x) <= tol).all()
        return
    y = np.clip(x / scale, -448, 448)
    err = 2.0 ** -22 * np.abs(y) + off / scale  # off, the fp32 reciprocal and the product
    grid = ref64.e4m3_values()
    i = np.clip(np.searchsorted(grid, np.abs(y)), 1, len(grid) - 1)
    best = np.minimum(np.abs(np.abs(y) - grid[i]), np.abs(np.abs(y) - grid[i - 1]))
    assert (np.abs(got - y) <= best + 2 * err).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_appended(case, decode, kind):
    from causal_gqa_attention_qkv_gb300 import attn, step
    case = case[:7] + (kind, case[8])
    _, _, d, _, _, sections, inter, _, _ = case
    w, host = make(case, decode)
    pos = positions(len(sections), w.num_tokens, seed=d + 3)
    rope = attn.RopeAxes(pos.cuda(), sections, inter)
    ds = step.upload(w, host)
    if decode:
        attn.decode(ds.cfg, ds.qkv, ds.q_norm_w, ds.k_norm_w, ds.max_cache_len, ds.kv_decode, ds.out, ds.workspace,
                    rope=rope)
    else:
        attn.kv_append(ds.cfg, ds.qkv, ds.k_norm_w, ds.cu_seqlens, ds.kv_prefill, ds.workspace, rope=rope)
    assert ds.status() == 0
    kv = ds.kv_prefill or ds.kv_decode
    _, k, v = ref64.prepared(w, host, (pos.numpy(), sections, inter))
    check_entries(kind, kv, host, "k", k, None if kind == "e2m1" else ref64.PAIR_REL * ref64.pair_norm(k))
    check_entries(kind, kv, host, "v", v, np.zeros_like(v))


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("d,axes", [(128, True), (64, True), (128, False)])
def test_projected(d, axes, kind):
    """The fused projection's K and V.  Its fp32 accumulation of C products is off by
    at most 1.5 C 2^-24 of their magnitudes' sum, a.  In K, w x / rms moves by at most
    w a / rms for x and w |x| a / rms^2 for the rms (w below 2), and a rotation turns
    the errors of two members into at most sqrt(2) of the larger."""
    from causal_gqa_attention_qkv_gb300 import attn, step
    hq, hkv, lens, cache, C = 8, 2, [130, 1, 65], [0, 40, 200], 256
    w = gen.custom(f"axst_{d}_{kind}", hq, hkv, d, lens, cache, seed=d)
    host = gen.make_inputs(w, kv_dtype=kind)
    assert float(host["k_norm_w"].abs().max()) < 2
    pj = gen.make_projection_inputs(w, hidden=C, seed=3)
    sections, n = [d // 2 - 20, 10, 10], w.num_tokens
    pos = positions(3, n, seed=8)
    ds = step.upload(w, host)
    q = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
    attn.qkv_proj_prepare(ds.cfg, pj["hidden"].cuda(), pj["w_qkv"].cuda(), ds.q_norm_w, ds.k_norm_w, ds.cu_seqlens,
                          ds.kv_prefill, q, ds.workspace, rope=attn.RopeAxes(pos.cuda(), sections, True) if axes else None)
    assert ds.status() == 0
    split = lambda t: t.numpy().reshape(n, hq + 2 * hkv, d)[:, hq:]
    x = split(pj["hidden"].double() @ pj["w_qkv"].double().T)
    acc = 1.5 * C * 2.0 ** -24 * split(pj["hidden"].double().abs() @ pj["w_qkv"].double().abs().T)
    at = ref64.places(host, d, (pos.numpy(), sections, True) if axes else None)
    k = ref64.norm_rope(x[:, :hkv], host["k_norm_w"].double().numpy(), at, w.rms_eps, w.rope_theta)
    rms = np.sqrt((x[:, :hkv] ** 2).mean(-1, keepdims=True))
    a = acc[:, :hkv].max(-1, keepdims=True) / rms
    off = ref64.PAIR_REL * ref64.pair_norm(k) + 2 * 2 ** 0.5 * a * (1 + np.abs(x[:, :hkv]).max(-1, keepdims=True) / rms)
    check_entries(kind, ds.kv_prefill, host, "k", k, off)
    check_entries(kind, ds.kv_prefill, host, "v", x[:, hkv:], acc[:, hkv:])
