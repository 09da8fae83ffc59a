"""GPU tests of the merge of a list's splits (block_merge of csrc/decode.cuh) from given partial
results: against the softmax of all of them, and with splits that gave up, whose lists are left
unwritten while the others are not.  The rest of attn_block_attend is in test_gpu_blocks.py."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
WARPS = 4


@pytest.fixture(scope="module")
def merge(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_gqa_attention_qkv_gb300 import build
    so = str(tmp_path_factory.mktemp("merge") / "block_merge.so")
    subprocess.check_call([build.NVCC, *build.ARCH, *build.FLAGS, "-shared", os.path.join(HERE, "block_merge.cu"), "-o", so])
    f = ctypes.CDLL(so).test_block_merge
    f.argtypes = [ctypes.c_int] * 5 + [ctypes.c_void_p] * 6
    return f


def run(merge, N, hkv, g, d, splits, gave_up, seed=0, none=0.1):
    """(out [N, hkv, g, d], what it has to be, what it may be off by); 776 where nothing is written."""
    rng = np.random.RandomState(seed)
    mo = rng.randn(N, hkv, splits, WARPS, g, d).astype(np.float32)
    mm = (4 * rng.randn(N, hkv, splits, WARPS, g)).astype(np.float32)
    ml = (1 + 9 * rng.rand(N, hkv, splits, WARPS, g)).astype(np.float32)
    empty = rng.rand(*mm.shape) < none  # a warp without a key
    mo[empty], mm[empty], ml[empty] = 0.0, -np.inf, 0.0
    dev = lambda x: torch.tensor(x).cuda()
    args = [dev(mo), dev(mm), dev(ml), dev(gave_up.astype(np.int32))]
    out = torch.full((N, hkv, g, d), 776.0, dtype=torch.bfloat16, device="cuda")
    rc = merge(N, hkv, g, d, splits, *[x.data_ptr() for x in args], out.data_ptr(),
               torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0
    o, m, l = mo.astype(np.float64), mm.astype(np.float64), ml.astype(np.float64)
    top = m.max((2, 3), keepdims=True)
    w = np.exp2(m - np.where(np.isinf(top), 0.0, top))
    total = (w * l).sum((2, 3))
    total = np.where(total == 0, 1.0, total)[..., None]
    want, size = ((w[..., None] * x).sum((2, 3)) / total for x in (o, np.abs(o)))
    # the output's rounding; two weights of 2^-21 each (a difference rounded before exp2, exp2 itself)
    # and fp32 sums of 64 terms at most, in the numerator and in the denominator: below 2^-17 of the magnitudes
    tol = 2.0 ** -8 * 1.01 * np.abs(want) + 2.0 ** -17 * size
    return out.double().cpu().numpy(), want, tol


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("splits", [1, 2, 3, 7, 8, 15, 16])
def test_merge_with_splits_that_gave_up(merge, splits, d):
    for g in (1, 3, 8):
        N, hkv = 5, 2
        gave_up = np.zeros((N, hkv, splits), bool)
        gave_up[1, 0, 0] = gave_up[2, 1, splits - 1] = gave_up[3, 0, splits // 2] = True
        gave_up[4, 1] = True
        out, want, tol = run(merge, N, hkv, g, d, splits, gave_up, seed=g)
        lost = gave_up.any(2)
        assert lost.sum() == 4 and (out[lost] == 776).all()
        assert (np.abs(out - want) <= tol)[~lost].all()


@pytest.mark.parametrize("splits", [1, 5, 16])
def test_merge_of_lists_that_leave_few_keys_or_none(merge, splits):
    for none in (0.9, 1.0):
        out, want, tol = run(merge, 4, 3, 4, 64, splits, np.zeros((4, 3, splits), bool), none=none)
        assert (np.abs(out - want) <= tol).all() and (none < 1.0 or (out == 0).all())
