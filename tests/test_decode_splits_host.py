"""CPU tests of the split counts and workspaces of decode calls whose splits are
longer: E2M1 caches and rotary axes."""
import ctypes

import pytest

from test_operators_host import FAKE, PAST_CHECKS, kv4, lib, rope  # noqa: F401 (lib is a fixture)

SIZES = [(1, 12), (1, 777), (3, 3000), (16, 65000), (37, 2500), (64, 1999), (64, 8192), (256, 16384), (4096, 300)]


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (8, 1, 64)])
@pytest.mark.parametrize("B,L", SIZES)
def test_splits_of_a_call(lib, B, L, hq, hkv, d):  # noqa: F811
    from causal_gqa_attention_qkv_gb300 import attn
    cfg = attn.config(hq, hkv, d)
    plain = attn.decode_splits(cfg, B, L)
    assert lib.attn_decode_splits(ctypes.byref(cfg), B, L) == plain
    assert attn.decode_splits(cfg, B, L, attn.ATTN_KV_E4M3) == plain
    longer = attn.decode_splits(cfg, B, L, attn.ATTN_KV_E2M1)
    for kind in (attn.ATTN_KV_BF16, attn.ATTN_KV_E4M3, attn.ATTN_KV_E2M1):
        assert attn.decode_splits(cfg, B, L, kind, axes=True) == longer
    assert 1 <= longer <= plain <= 16
    # every split but the last holds at least min(2048, 8 B Hkv) keys
    assert (longer - 1) * min(2048, 8 * B * hkv) < L + 1


def test_bad_arguments(lib):  # noqa: F811
    from causal_gqa_attention_qkv_gb300 import attn
    c = ctypes.byref(attn.config(32, 8, 128))
    for args in ((None, 1, 5, 0, 0), (c, -1, 5, 0, 0), (c, 1, -1, 0, 0), (c, 1, 5, 3, 0), (c, 1, 5, -1, 1)):
        assert lib.attn_decode_splits_of(*args) == -1
    with pytest.raises(attn.AttnError):
        attn.decode_splits(attn.config(32, 8, 128), 1, 5, 7)


@pytest.mark.parametrize("B,L", SIZES)
def test_a_call_asks_for_the_workspace_it_uses(lib, B, L):  # noqa: F811
    from causal_gqa_attention_qkv_gb300 import attn
    f, cfg = ctypes.c_void_p(FAKE), attn.config(32, 8, 128)
    c, up = ctypes.byref(cfg), lambda x: -(-x // 256) * 256
    r = ctypes.byref(rope(attn, ld=B))
    for kind, axes in ((0, None), (1, None), (2, None), (0, r), (1, r), (2, r)):
        k = ctypes.byref(kv4(attn, kv_dtype=kind))
        n = attn.decode_splits(cfg, B, L, kind, axes is not None)
        rows = B * 32 * n
        need = 256 + (up(rows * 128 * 4) + up(rows * 8) if n > 1 else 0)
        assert need <= attn.workspace_size(cfg, 0, B, L + 1)
        for size, ok in ((need, True), (need - 256, False)):
            for rc in (lib.attn_decode_axes(c, f, f, f, B, L, k, axes, f, f, size, None),
                       lib.attn_decode_attend_axes(c, f, f, B, L, k, axes, f, f, size, None)):
                assert (rc in PAST_CHECKS) if ok else rc == -3, (kind, size, rc)
