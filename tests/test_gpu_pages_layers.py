"""GPU test of one pool that holds the pages of several layers: layer l of request b
is row l * requests + b of the table, so every page call takes all layers at once
and a layer's calls see the rows of that layer."""
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


@pytest.mark.parametrize("kind", ["bf16", "e2m1"])
def test_serving_loop_of_three_layers(kind):
    from causal_gqa_attention_qkv_gb300 import attn
    L, B, hq, hkv, d, ps, ppr = 3, 4, 4, 2, 128, 64, 5
    S = ppr * ps
    pool = Pool(kind, 50, ps, hkv, d, [], L * B, ppr, seed=7)
    cfg, kv, ref, ws = attn.config(hq, hkv, d), pool.kv, pool.ref, pool.ws
    W = (hq + 2 * hkv) * d
    g = torch.Generator().manual_seed(13)
    nw = [[(1 + 0.1 * torch.randn(d, generator=g)).bfloat16().cuda() for _ in range(2)] for _ in range(L)]
    new = lambda n: torch.randn(n, W, generator=g).bfloat16().cuda()
    empty = lambda n: torch.empty(n, hq * d, dtype=torch.bfloat16, device="cuda")
    aws = attn.new_workspace(cfg, 256, B, S)
    rows = lambda bs: i32([l * B + b for l in range(L) for b in bs])
    each = lambda ns: i32(list(ns) * L)

    # the same layers, each in a contiguous cache of its own
    def flat_cache():
        like = lambda t: torch.zeros(B * S, *t.shape[1:], dtype=t.dtype, device="cuda")
        blocks = [torch.zeros(hkv, B * S, d // 16, dtype=torch.uint8, device="cuda") if kind == "e2m1" else None
                  for _ in range(2)]
        return attn.KVCache(like(kv.k_cache), like(kv.v_cache), torch.arange(0, B * S, S, device="cuda"),
                            torch.zeros(B, dtype=torch.int32, device="cuda"), i32([S] * B), None, 0, 0.03, 0.06, *blocks)

    flat = [flat_cache() for _ in range(L)]

    def flat_fork(s, t):
        for f in flat:
            for x in (f.k_cache, f.v_cache):
                x[t * S:t * S + S] = x[s * S:s * S + S].clone()
            for x in (f.k_block_scale, f.v_block_scale):
                if x is not None:
                    x[:, t * S:t * S + S] = x[:, s * S:s * S + S].clone()
            f.cache_lens[t] = f.cache_lens[s]

    lens = [100, 64]
    attn.pages_reserve(kv, ref, rows([0, 1]), each(lens), ws)
    for l in range(L):
        x, out, want = new(164), empty(164), empty(164)
        attn.prefill(cfg, x, *nw[l], i32([0, 100, 164]), 100, kv.rows(l * B, l * B + 2), out, aws)
        attn.prefill(cfg, x, *nw[l], i32([0, 100, 164]), 100, flat[l].rows(0, 2), want, aws)
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
        kv.cache_lens[l * B:l * B + 2] += i32(lens)
        flat[l].cache_lens[:2] += i32(lens)

    def decode(steps):
        for _ in range(steps):
            attn.pages_reserve(kv, ref, rows(range(B)), each([1] * B), ws)
            for l in range(L):
                x, out, want = new(B), empty(B), empty(B)
                attn.decode(cfg, x, *nw[l], S - 1, kv.rows(l * B, l * B + B), out, aws)
                attn.decode(cfg, x, *nw[l], S - 1, flat[l], want, aws)
                assert torch.equal(out.view(torch.int16), want.view(torch.int16))
                flat[l].cache_lens += 1
            kv.cache_lens += 1

    attn.pages_fork(cfg, kv, ref, rows([0, 0]), rows([2, 3]), ws)  # all layers of both forks in one call
    flat_fork(0, 2)
    flat_fork(0, 3)
    decode(35)
    attn.pages_free(kv, ref, rows([0, 3]), ws)
    attn.pages_compact(cfg, kv, ref, ws)  # moves every layer's pages, by one plan
    used = int((ref > 0).sum())
    assert (ref[:used] > 0).all() and (ref[used:] == 0).all()
    attn.pages_fork(cfg, kv, ref, rows([1, 2]), rows([0, 3]), ws)
    flat_fork(1, 0)
    flat_fork(2, 3)
    decode(10)
    attn.pages_free(kv, ref, rows(range(B)), ws)
    assert (ref == 0).all() and (kv.page_table == -1).all()
    assert attn.get_status(ws) == 0 and attn.get_status(aws) == 0
