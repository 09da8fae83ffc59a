"""CPU tests of the check that a call's cfg is that of its cache: refused before a
tensor's address is taken."""
import pytest
import torch

from causal_gqa_attention_qkv_gb300 import attn


def cache(kind, S=128, H=4, D=64, flat=False):
    row = D // 2 if kind == "e2m1" else D
    k = torch.zeros(S, H, row, dtype=torch.bfloat16 if kind == "bf16" else torch.uint8)
    k = k.view(S, H * row) if flat else k
    blocks = [torch.zeros(H, S, D // 16, dtype=torch.uint8) for _ in range(2)] if kind == "e2m1" else [None, None]
    i32 = torch.zeros(2, dtype=torch.int32)
    return attn.KVCache(k, k.clone(), i32.long(), i32, i32, torch.zeros(2, 1, dtype=torch.int32), 64, 1.0, 1.0, *blocks)


def refused(kv, cfg, exact):
    with pytest.raises(AssertionError) as e:  # CPU tensors: a cfg that fits is refused later, for its tensors
        kv.struct_for(cfg, exact)
    return "cfg" in str(e.value)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e2m1"])
def test_another_cfg_is_refused(kind):
    kv = cache(kind)
    fits, wide, long, swapped, narrow = (attn.config(*x) for x in ((8, 4, 64), (8, 8, 64), (8, 4, 128), (8, 2, 128),
                                                                   (8, 2, 64)))
    for exact in (False, True):
        assert not refused(kv, fits, exact)
        assert refused(kv, wide, exact) and refused(kv, long, exact)      # past the end
        assert refused(kv, swapped, exact) == (kind == "e2m1")           # the same bytes; scales lie elsewhere
        assert refused(kv, narrow, exact) == (kind == "e2m1" or exact)
    kv.v_cache = kv.v_cache[:64]
    assert refused(kv, fits, True) or kind == "e2m1"  # (of an E2M1 cache the struct compares both)


def test_a_flat_view_of_the_slots_stays_accepted():
    assert not refused(cache("bf16", flat=True), attn.config(8, 4, 64), False)
    assert not refused(cache("bf16", flat=True), attn.config(8, 4, 64), True)


@pytest.mark.parametrize("kind", ["bf16", "e2m1"])
@pytest.mark.parametrize("heads", [(8, 3, 64), (8, 16, 64), (8, 4, 96), (256, 128, 128)])
def test_a_cfg_that_the_library_refuses_is_left_to_it(kind, heads):
    """Its own code (ATTN_EINVAL, ATTN_EGQA) reaches the caller, as for calls without a cache."""
    from causal_gqa_attention_qkv_gb300 import build
    build.build()
    assert not refused(cache(kind), attn.config(*heads), True)
