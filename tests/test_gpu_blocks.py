"""GPU tests of the block calls (include/blocks.h): bounds, selection and attention over
lists against the plain 64-bit forms, for all cache types, layouts and head shapes, at
the sizes and lists where they can go wrong; then a served batch that uses them
together, eager and captured."""
import numpy as np
import pytest
import torch

import ref_blocks as rb
from ref_blocks import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_gqa_attention_qkv_gb300 import build
    build.build()


def status(ws):
    from causal_gqa_attention_qkv_gb300 import attn
    return attn.get_status(ws)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


KINDS = ("bf16", "e4m3", "e2m1")
CAP, SEQ, BOUNDS = 1, 2, 8


# ------------------------------------------------------------------ bounds
def check_bounds(s, start=None, cu=True):
    from causal_gqa_attention_qkv_gb300 import attn
    ws = s.workspace(1)
    before = s.bounds.clone()
    attn.block_bounds(s.cfg, s.kv, s.blocks, s.cu if cu else None, ws, start=None if start is None else i32(start))
    assert status(ws) == 0
    want = before.double().cpu().numpy()
    for row, v in rb.bounds(s.c, s.entries("k"), start).items():
        want[row] = v
    assert np.array_equal(s.bounds.double().cpu().numpy(), want)
    return (want != before.double().cpu().numpy()).any()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page,block", [(0, 64), (64, 64), (128, 64), (256, 128), (256, 256), (0, 256), (1024, 128)])
@pytest.mark.parametrize("d,hkv", [(128, 8), (64, 3)])
def test_bounds(kind, page, block, d, hkv):
    cached, new = [0, 63, 64, 511, 200, 1000], [1, 1, 64, 300, 0, 777]
    s = Cache(kind, hkv, hkv, d, cached, new, page, block, seed=page + block)
    assert check_bounds(s)
    assert check_bounds(s, start=[0, -9, 100, 0, 64, 900])


@pytest.mark.parametrize("kind", KINDS)
def test_bounds_of_single_tokens(kind):
    """cu_seqlens None: one new token per request; only blocks that become full are made."""
    cached = [63, 64, 0, 127, 191, 126]
    s = Cache(kind, 4, 2, 64, cached, [1] * 6, 64, 64)
    assert check_bounds(s, cu=False)
    assert (s.bounds == 776).all(-1).all(-1).all(-1).sum() == s.c["rows"] - 3


def test_bounds_of_many_requests_and_long_ones():
    s = Cache("bf16", 1, 1, 64, [i % 130 for i in range(1500)], [1 + i % 3 for i in range(1500)], 64, 64)
    assert check_bounds(s)
    s = Cache("e2m1", 2, 2, 128, [0], [70001], 0, 256)
    assert check_bounds(s)


def test_bounds_of_entries_that_are_not_finite():
    s = Cache("bf16", 2, 2, 64, [0], [256], 64, 64)
    k = s.kv.k_cache
    at = lambda p: int(rb.slots_of(s.c, 0, [p])[0])
    k[at(3), 0, 5] = float("nan")
    k[at(70), 1, 0] = float("inf")
    k[at(130), 0, 7] = float("-inf")
    from causal_gqa_attention_qkv_gb300 import attn
    ws = s.workspace(1)
    attn.block_bounds(s.cfg, s.kv, s.blocks, s.cu, ws)
    got = s.bounds.double().cpu().numpy()
    want = rb.bounds(s.c, s.entries("k"))
    for row, v in want.items():
        assert np.array_equal(got[row], v, equal_nan=True)
    assert np.isnan(got[rb.row_of(s.c, 0, 0), 0, :, 5]).all() and got[rb.row_of(s.c, 0, 1), 1, 1, 0] == np.inf


@pytest.mark.parametrize("code", [0x7F, 0xFF])
def test_bounds_of_code_that_is_no_number(code):
    s = Cache("e4m3", 2, 2, 64, [0], [128], 0, 64)
    s.kv.k_cache[int(s.c["base"][0]) + 10, 1, 3] = code
    from causal_gqa_attention_qkv_gb300 import attn
    attn.block_bounds(s.cfg, s.kv, s.blocks, s.cu, s.workspace(1))
    got = s.bounds[rb.row_of(s.c, 0, 0)].float()
    assert got[1, :, 3].isnan().all() and int(got.isnan().sum()) == 2


@pytest.mark.parametrize("kind,page,block", [("e4m3", 64, 64), ("e2m1", 256, 128), ("e4m3", 0, 256), ("e2m1", 0, 64)])
@pytest.mark.parametrize("scale", [0.037, 1 / 3, 1e-38, 2.5e37])
def test_bounds_under_scales_that_round(kind, page, block, scale):
    """k_scale no power of two: the bounds are those of the entries that attn_kv_gather gives, bit for
    bit, and the score bounds q . k of those; of the codes' own values it does to within 2^-8 of the
    products' magnitudes, which rounding an entry to bf16 moves by at most that."""
    import ref64
    from causal_gqa_attention_qkv_gb300 import attn
    scale = float(np.float32(scale))
    s = Cache(kind, 4, 2, 64, [0, 100], [700, 413], page, block, seed=block)
    s.kv.k_scale = scale
    ws = s.workspace(1)
    attn.block_bounds(s.cfg, s.kv, s.blocks, s.cu, ws, start=i32([0, 0]))
    assert status(ws) == 0
    exact = ref64.entries(s.kv.k_cache, kind, scale, s.kv.k_block_scale)
    got = s.bounds.double().cpu().numpy()
    want = rb.bounds(s.c, exact, [0, 0])
    assert len(want) == 700 // block + 513 // block
    for row in range(s.c["rows"]):
        assert np.array_equal(got[row], want.get(row, np.full_like(got[row], 776.0)))
    k = [torch.empty(700 + 513, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    s.kv.cache_lens.copy_(i32([700, 513]))  # all entries are cached by now
    attn.kv_gather(s.cfg, s.kv, i32([0, 700, 1213]), i32([0, 0]), *k, ws)
    assert status(ws) == 0
    read = k[0].double().cpu().numpy()
    q = np.random.RandomState(1).randn(2, 2, 64)  # [Hkv, G, D]
    for b, at, n in ((0, 0, 700), (1, 700, 513)):
        for i in range(n // block):
            row, here = rb.row_of(s.c, b, i), slice(at + i * block, at + (i + 1) * block)
            own = exact[rb.slots_of(s.c, b, np.arange(i * block, (i + 1) * block))]
            assert np.array_equal(got[row], np.stack((read[here].min(0), read[here].max(0)), 1))
            if scale > 1 or scale < 1e-30:  # overflow, or steps that are no longer relative
                continue
            for h in range(2):
                top = rb.score(q[h], got[row, h, :1], got[row, h, 1:])[0]
                for keys, off in ((read[here, h], 0.0), (own[:, h], 2.0 ** -8)):
                    dots = (keys @ q[h].T).sum(1)
                    slack = off * (np.abs(keys) @ np.abs(q[h]).T).sum(1)
                    assert (top >= dots - slack - 1e-12 * np.abs(top)).all()


def test_bounds_problems_set_the_status():
    from causal_gqa_attention_qkv_gb300 import attn
    s = Cache("bf16", 2, 2, 64, [0, 0, 100], [200, 200, 30], 64, 64)
    ws = s.workspace(1)
    s.kv.page_table[0, 1] = 10 ** 6  # a page outside the cache: no row for its block
    s.kv.slot_capacity[1] = 199      # a region that is too small: skipped
    s.c["table"][0, 1] = 10 ** 6
    s.c["new"][1] = 0
    attn.block_bounds(s.cfg, s.kv, s.blocks, s.cu, ws)
    assert status(ws) == CAP
    want = rb.bounds(s.c, s.entries("k"))
    got = s.bounds.double().cpu().numpy()
    for row in range(s.c["rows"]):
        assert np.array_equal(got[row], want.get(row, np.full_like(got[row], 776.0)))
    # contiguous: rows behind the bounds are not written
    s = Cache("bf16", 2, 2, 64, [0], [256], 0, 64)
    ws = s.workspace(1)
    s.blocks.row_base = torch.tensor([s.c["rows"] - 2]).cuda()
    s.c["row_base"] = np.array([s.c["rows"] - 2])
    attn.block_bounds(s.cfg, s.kv, s.blocks, s.cu, ws)
    assert status(ws) == CAP
    want = rb.bounds(s.c, s.entries("k"))
    assert len(want) == 2
    for row, v in want.items():
        assert np.array_equal(s.bounds[row].double().cpu().numpy(), v)


# ------------------------------------------------------------------ selection
def fill_bounds(s, seed=0):
    rng = torch.Generator().manual_seed(seed)
    shape = (s.c["rows"], s.hkv, s.d)
    mid, half = torch.randn(shape, generator=rng), 1 + torch.rand(shape, generator=rng)
    s.bounds.copy_(torch.stack((mid - half, mid + half), 2).bfloat16())


def run_select(s, first, last, keep, cu=True, max_len=None):
    from causal_gqa_attention_qkv_gb300 import attn
    ws = s.workspace(keep, max_len)
    lists = torch.full((s.N, s.hkv, keep), -7, dtype=torch.int32, device="cuda")
    attn.block_select(s.cfg, s.q, s.cu if cu else None, s.max_len if max_len is None else max_len, s.kv, s.blocks, first,
                      last, lists, ws)
    return lists.cpu().numpy(), status(ws)


FORMS = (None, 1 << 20)  # bounds on the lengths: with the second, scores go through the workspace


def check_select(s, first, last, keep, cu=True, max_len=None):
    want = rb.select(s.c, s.q64(), s.bounds.double().cpu().numpy(), first, last, keep)
    for bound in FORMS if max_len is None else (max_len,):
        got, st = run_select(s, first, last, keep, cu, bound)
        assert st == 0
        assert np.array_equal(got, want)


@pytest.mark.parametrize("kind,hq,hkv,d", [("bf16", 8, 2, 128), ("e4m3", 8, 8, 64), ("e2m1", 16, 2, 128), ("bf16", 8, 1, 64),
                                           ("e4m3", 6, 3, 128)])
@pytest.mark.parametrize("page,block", [(0, 64), (64, 64), (256, 128), (128, 64), (256, 256)])
def test_select_single_tokens(kind, hq, hkv, d, page, block):
    cached = [0, 1, 63, 64, 64 * 7 - 1, 5000, 2047, 777, 20000]
    s = Cache(kind, hq, hkv, d, cached, [1] * len(cached), page, block, seed=hq + block)
    fill_bounds(s)
    for first, last, keep in ((1, 2, 8), (0, 1, 5), (2, 2, 4), (0, 1, 1), (3, 5, 60), (0, 1, 400)):
        check_select(s, first, last, keep, cu=keep != 60)


@pytest.mark.parametrize("kind,hq,hkv,d", [("bf16", 8, 2, 128), ("e2m1", 4, 4, 64)])
@pytest.mark.parametrize("page,block", [(0, 64), (128, 128)])
def test_select_several_tokens(kind, hq, hkv, d, page, block):
    """Runs of tokens that cross a block's end, groups of eight, requests without tokens."""
    cached, new = [60, 3000, 0, 5000, 127, 900], [9, 1, 40, 17, 0, 8]
    s = Cache(kind, hq, hkv, d, cached, new, page, block, seed=5)
    fill_bounds(s)
    for first, last, keep in ((1, 2, 8), (0, 1, 3), (1, 1, 2)):
        check_select(s, first, last, keep)


@pytest.mark.parametrize("hq,hkv", [(3, 3), (6, 3), (4, 1), (24, 3)])
@pytest.mark.parametrize("new", [1, 6])
def test_select_for_groups_of_any_size(hq, hkv, new):
    s = Cache("bf16", hq, hkv, 64, [3000, 900, 64 * 64], [new] * 3, 64, 64, seed=hq)
    fill_bounds(s)
    for first, last, keep in ((1, 1, 12), (0, 1, 2)):
        check_select(s, first, last, keep)


@pytest.mark.parametrize("new", [1, 6])
def test_blocks_of_no_page_count_as_zero(new):
    s = Cache("bf16", 8, 2, 128, [3000, 2000], [new, new], 128, 64, seed=3)
    fill_bounds(s)
    zero = s.bounds.double().cpu().numpy()
    for b, page, bad in ((0, 3, -1), (0, 11, 10 ** 6), (1, 7, -2 ** 31), (0, 17, s.c["slots"] // 128)):
        row = int(s.c["table"][b, page]) * 2
        zero[row:row + 2] = 0.0
        s.kv.page_table[b, page] = bad
    for bound in FORMS:
        got, st = run_select(s, 1, 1, 9, max_len=bound)
        assert st == CAP
        assert np.array_equal(got, rb.select(s.c, s.q64(), zero, 1, 1, 9))


@pytest.mark.parametrize("base", [-2 ** 33 + 5, -2 ** 40, 2 ** 33 + 1, -1000, 2 ** 62])
@pytest.mark.parametrize("new", [1, 6])
def test_rows_far_outside_the_bounds(base, new):
    """None of them is read: every block counts as 0, and ties go to the lower ones."""
    s = Cache("bf16", 8, 2, 128, [3000], [new], 0, 64)
    fill_bounds(s)
    s.blocks.row_base = torch.tensor([base]).cuda()
    n = [(3000 + j) // 64 + 1 for j in range(new)]
    want = np.array([list(range(7)) + [k - 2, k - 1] for k in n])
    for bound in FORMS:
        got, st = run_select(s, 1, 2, 9, max_len=bound)
        assert st == CAP
        assert np.array_equal(got, np.repeat(want[:, None], 2, 1))


def lattice_bounds(s, step, seed=0):
    """Bounds whose scores are multiples of a small step: many are equal, or a step apart."""
    rng = torch.Generator().manual_seed(seed)
    mid = torch.randint(-3, 4, (s.c["rows"], s.hkv, s.d), generator=rng).float()
    s.bounds.copy_(torch.stack((mid - 1, mid + 1), 2).bfloat16())
    s.bounds[:, :, 0, 0] = (-step * torch.randint(0, 3, (s.c["rows"], s.hkv), generator=rng)).bfloat16().cuda()


@pytest.mark.parametrize("step", [0.0, 2.0 ** -9, 2.0 ** -30])
@pytest.mark.parametrize("new", [1, 6])
def test_scores_that_are_close_around_the_last_one_taken(step, new):
    s = Cache("bf16", 8, 2, 128, [64 * 120, 64 * 300 + 5], [new, new], 0, 64, seed=int(step * 512))
    s.q.copy_(torch.randint(-2, 3, s.q.shape, generator=torch.Generator().manual_seed(1)).to(s.q))
    lattice_bounds(s, step)
    for keep in (2, 3, 7, 20, 64, 100):
        check_select(s, 0, 1, keep)


def test_select_many_requests():
    s = Cache("bf16", 2, 1, 64, [700 + 3 * i for i in range(700)], [1] * 700, 64, 64)
    fill_bounds(s)
    check_select(s, 1, 1, 6, cu=True)
    check_select(s, 1, 1, 6, cu=False)
    s = Cache("bf16", 2, 1, 64, [900 + i for i in range(300)], [i % 5 for i in range(300)], 64, 64)
    fill_bounds(s)
    check_select(s, 1, 1, 6)


@pytest.mark.parametrize("batch,new", [(1, 1), (2, 1), (9, 1), (16, 1), (48, 1), (49, 1), (10, 3), (24, 2), (25, 2), (20, 3),
                                       (2, 24), (1, 50)])
@pytest.mark.parametrize("blocks", [31, 33, 70, 140, 300, 1030])
def test_select_around_the_choice_of_kernels(batch, new, blocks):
    """Numbers of lists and candidates where the split over CTAs changes."""
    s = Cache("bf16", 4, 2, 64, [64 * blocks - 1 - i % 7 for i in range(batch)], [new] * batch, 0, 64, seed=blocks)
    fill_bounds(s)
    check_select(s, 1, 1, 9)


@pytest.mark.parametrize("cached", [64 * 2047, 64 * 2048 + 5, 64 * 2050, 64 * 5000])
def test_select_of_long_requests(cached):
    """Around the number of candidates that one kernel takes, and past it."""
    s = Cache("bf16", 4, 1, 64, [cached, 70], [1, 1], 0, 64)
    fill_bounds(s)
    for first, last, keep in ((0, 1, 33), (1, 2, 2000), (0, 1, 4096)):
        check_select(s, first, last, keep)


def test_select_over_a_loose_host_bound():
    s = Cache("bf16", 8, 2, 128, [3000, 100], [1, 1], 64, 64)
    fill_bounds(s)
    check_select(s, 1, 1, 9, max_len=60000)
    check_select(s, 1, 1, 9, max_len=1 << 24)


@pytest.mark.parametrize("cached,new", [([64 * 300] * 3, [1] * 3), ([64 * 300, 64 * 40], [5, 20]), ([64 * 3000], [1])])
def test_equal_scores_go_to_the_lower_block(cached, new):
    s = Cache("bf16", 4, 2, 64, cached, new, 0, 64)
    s.bounds.zero_()
    check_select(s, 1, 2, 20)
    fill_bounds(s)
    s.bounds[:] = s.bounds[3].clone()
    check_select(s, 1, 2, 20)
    s.bounds[::3] = s.bounds[0] * 1.5  # two values only
    check_select(s, 0, 1, 50)
    fill_bounds(s, 1)
    s.q.zero_()
    check_select(s, 0, 1, 17)


@pytest.mark.parametrize("new", [1, 3])
def test_scores_that_fp32_sums_cannot_tell_apart(new):
    """Scores that differ by far less than the rounding of their sums: large products that
    cancel, and a small one that decides."""
    s = Cache("bf16", 1, 1, 64, [64 * 500], [new], 0, 64)
    s.q.fill_(1.0)
    s.bounds.zero_()
    rng = np.random.RandomState(0)
    n = s.c["rows"]
    big = torch.tensor(rng.choice([2.0 ** 20, 2.0 ** 19, 3.0 * 2 ** 18], n)).cuda()
    for a, b in ((0, 1), (8, 17), (30, 63)):
        s.bounds[:, 0, 1, a], s.bounds[:, 0, 1, b] = big.bfloat16(), -big.bfloat16()
    s.bounds[:, 0, 1, 5] = torch.tensor(rng.permutation(n) % 251 * 2.0 ** -9).cuda().bfloat16()
    check_select(s, 0, 1, 40)
    check_select(s, 1, 3, 300)


def test_scores_in_a_crowd_beside_outliers():
    """One score far from all others: the bins of equal width hold hundreds of keys in one."""
    for far in (3e30, -3e30):
        s = Cache("bf16", 2, 1, 64, [64 * 1500], [1], 0, 64)
        fill_bounds(s)
        s.bounds.mul_(2.0 ** -20)
        s.bounds[700] = far
        check_select(s, 0, 1, 64)
        s.bounds[700:720] = s.bounds[720:740] * 1e25
        check_select(s, 1, 1, 30)


def test_bounds_that_are_not_finite_rank_as_stated():
    s = Cache("bf16", 4, 2, 64, [64 * 200], [1], 0, 64)
    fill_bounds(s)
    base = int(s.c["row_base"][0])
    s.bounds[base + 50, 0, 0, 3] = float("nan")
    s.bounds[base + 60, 1, 1, 9] = float("inf")
    s.bounds[base + 61, 1, 0, 9] = float("-inf")
    s.bounds[base + 62, 1, 1, 4] = float("-inf")
    s.q[0, :, 9] = 1.0  # M is 0 there: 0 * -inf is no number
    s.q[0, :, 4] = torch.tensor([1.0, -1.0, 2.0, 0.5])
    check_select(s, 0, 1, 12)
    got, _ = run_select(s, 0, 1, 12)
    assert 50 in got[0, 0] and 60 in got[0, 1] and 61 in got[0, 1]
    s.q[0, 2, 0] = float("nan")
    check_select(s, 0, 1, 12)


@pytest.mark.parametrize("new", [1, 3])
def test_scores_beyond_fp32(new):
    s = Cache("bf16", 4, 1, 128, [64 * 300], [new], 0, 64)
    fill_bounds(s)
    s.bounds.mul_(1e37)
    s.q.mul_(1e3)
    check_select(s, 0, 1, 25)
    fill_bounds(s)
    s.bounds.mul_(1e-38)
    s.q.mul_(1e-6)
    check_select(s, 0, 1, 25)
    s.q.fill_(3.0)  # subnormal bounds, which a tensor core may take for zeros
    check_select(s, 0, 1, 25)
    s.q[:, 1].fill_(3.38e38)  # a coefficient next to the largest number
    check_select(s, 0, 1, 25)


def test_select_problems_set_the_status():
    s = Cache("bf16", 2, 1, 64, [3000, 5000, 2000], [2, 2, 2], 64, 64)
    fill_bounds(s)
    # a host bound below the second request: its lists stay unwritten
    got, st = run_select(s, 1, 1, 6, max_len=4000)
    want = rb.select(s.c, s.q64(), s.bounds.double().cpu().numpy(), 1, 1, 6)
    assert st == BOUNDS and (got[2:4] == -7).all() and np.array_equal(got[[0, 1, 4, 5]], want[[0, 1, 4, 5]])
    # a page outside the cache reads as zeros
    s.kv.page_table[2, 7] = -1
    s.c["table"][2, 7] = -1
    got, st = run_select(s, 1, 1, 6)
    assert st == CAP
    assert np.array_equal(got, rb.select(s.c, s.q64(), s.bounds.double().cpu().numpy(), 1, 1, 6))
    # a region that is too small
    s.kv.slot_capacity[0] = 3001
    got, st = run_select(s, 1, 1, 6)
    assert st == CAP and (got[:2] == -7).all() and (got[2:] != -7).all()
    # tokens behind the last request
    s.cu[3] = 5
    got, st = run_select(s, 1, 1, 6)
    assert st & SEQ and (got[5] == -7).all()


@pytest.mark.parametrize("new", [1, 8])
def test_a_request_one_position_past_the_host_bound(new):
    """None of its lists is written, those of tokens before the bound and of a bound within the
    last block among them; at the bound all are."""
    s = Cache("bf16", 2, 1, 64, [3005, 64 * 40 - 3 - new, 1000], [new] * 3, 64, 64)
    fill_bounds(s)
    want = rb.select(s.c, s.q64(), s.bounds.double().cpu().numpy(), 1, 1, 6)
    got, st = run_select(s, 1, 1, 6, max_len=3005 + new)
    assert st == 0 and np.array_equal(got, want)
    got, st = run_select(s, 1, 1, 6, max_len=3005 + new - 1)
    assert st == BOUNDS and (got[:new] == -7).all() and np.array_equal(got[new:], want[new:])
    # the same in the two-kernel form (more tokens per request)
    s = Cache("bf16", 4, 4, 64, [3005, 64 * 40 - 3 - 9 * new], [9 * new, 9 * new], 0, 64)
    fill_bounds(s)
    want = rb.select(s.c, s.q64(), s.bounds.double().cpu().numpy(), 1, 1, 6)
    got, st = run_select(s, 1, 1, 6, max_len=3005 + 9 * new - 1)
    assert st == BOUNDS and (got[:9 * new] == -7).all() and np.array_equal(got[9 * new:], want[9 * new:])


@pytest.mark.parametrize("B", [3, 40, 300])
@pytest.mark.parametrize("form", ["up and down", "steps of 2^31 - 1", "backwards", "one far too long", "negative"])
def test_seqlens_that_are_in_no_order(B, form):
    """Reported, and no list holds anything but blocks of a request; a batch after it is as ever."""
    s = Cache("bf16", 4, 4, 64, [64 * 50 + i % 60 for i in range(B)], [3] * B, 0, 64)
    fill_bounds(s)
    want = rb.select(s.c, s.q64(), s.bounds.double().cpu().numpy(), 1, 1, 6)
    cu, n = s.cu.clone(), np.arange(B + 1)
    big = 2 ** 31 - 1
    s.cu.copy_(i32({"up and down": np.where(n % 2, s.N, 0), "steps of 2^31 - 1": np.where(n % 2, big, 0),
                    "backwards": 3 * (B - n), "one far too long": np.where(n == B, big, 3 * n),
                    "negative": np.where(n % 2, big - 8, -big + n)}[form]))
    for bound in FORMS:
        got, st = run_select(s, 1, 1, 6, max_len=bound)
        assert st and ((got >= 0) & (got < 52) | (got == -7)).all()
    s.cu.copy_(cu)
    for bound in FORMS:
        got, st = run_select(s, 1, 1, 6, max_len=bound)
        assert st == 0 and np.array_equal(got, want)


def test_select_over_rows_past_two_to_the_31_bytes():
    """Bounds of more than 4 GB: rows are found by 64-bit offsets."""
    s = Cache("bf16", 8, 8, 128, [64 * 90], [1], 0, 64)
    rows = (5 << 30) // (8 * 2 * 128 * 2)
    s.bounds = torch.zeros(rows, 8, 2, 128, dtype=torch.bfloat16, device="cuda")
    at = rows - 95
    s.blocks.bounds, s.blocks.row_base = s.bounds, torch.tensor([at]).cuda()
    s.bounds[at:at + 91] = torch.randn(91, 8, 2, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    ref = dict(s.c, row_base=np.array([0]), rows=91)
    got, st = run_select(s, 1, 1, 8)
    assert st == 0
    assert np.array_equal(got, rb.select(ref, s.q64(), s.bounds[at:at + 91].double().cpu().numpy(), 1, 1, 8))


# ------------------------------------------------------------------ attention over lists
def random_lists(s, keep, seed=0, forms=True):
    """Lists of blocks in any order, with holes, blocks past the query, and one block twice."""
    rng = np.random.RandomState(seed)
    lists = np.full((s.N, s.hkv, keep), -1, np.int32)
    t = 0
    for cached, new in zip(s.c["cached"], s.c["new"]):
        for j in range(new):
            n = (cached + j) // s.c["block"] + 1
            for h in range(s.hkv):
                m = min(keep, n)
                lists[t, h, :m] = rng.permutation(n)[:m]
                form = rng.randint(6) if forms else 0
                if form == 1:
                    lists[t, h, rng.randint(keep)] = -1 - rng.randint(5)
                elif form == 2:
                    lists[t, h, rng.randint(keep)] = n + rng.randint(3) * 10 ** 6
                elif form == 3:
                    lists[t, h, -1] = lists[t, h, 0]
                elif form == 4:
                    lists[t, h] = rng.permutation(lists[t, h])
            t += 1
    return lists


def run_attend(s, lists, cu=True):
    from causal_gqa_attention_qkv_gb300 import attn
    ws = s.workspace(lists.shape[2])
    out = torch.full((s.N, s.hq * s.d), 776.0, dtype=torch.bfloat16, device="cuda")
    attn.block_attend(s.cfg, s.q, s.cu if cu else None, s.kv, s.c["block"], i32(lists), out, ws)
    return out.double().cpu().numpy().reshape(s.N, s.hq, s.d), status(ws)


def check_attend(s, lists, cu=True):
    out, st = run_attend(s, lists, cu)
    assert st == 0
    want, tol = rb.attend(s.c, s.q64(), lists, s.entries("k"), s.entries("v"), s.kind != "bf16")
    off = np.abs(out - want)
    assert (off <= tol).all(), (off - tol).max()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (8, 8, 64), (8, 1, 128), (16, 2, 64), (6, 3, 128)])
@pytest.mark.parametrize("page,block", [(0, 64), (64, 64), (256, 128), (256, 256)])
def test_attend(kind, hq, hkv, d, page, block):
    cached, new = [0, 63, 64, 700, 5000, 129], [1, 1, 2, 5, 1, 0]
    s = Cache(kind, hq, hkv, d, cached, new, page, block, seed=hq + page)
    check_attend(s, random_lists(s, 7))
    check_attend(s, random_lists(s, 1, seed=1))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("batch,keep", [(1, 64), (1, 65), (3, 40), (20, 17), (100, 3), (1, 300)])
def test_attend_single_tokens_over_splits(kind, batch, keep):
    """Lists that are cut into 1 to 16 parts, of equal and unequal length."""
    cached = [20000 + 77 * i if keep > 3 else 300 + i for i in range(batch)]
    s = Cache(kind, 8, 2, 64, cached, [1] * batch, 64, 64, seed=keep)
    check_attend(s, random_lists(s, keep, forms=batch > 1), cu=False)


@pytest.mark.parametrize("kind", KINDS)
def test_attend_with_the_longest_lists(kind):
    s = Cache(kind, 2, 1, 64, [64 * 5000], [1], 0, 64)
    lists = random_lists(s, 4096, forms=False)
    check_attend(s, lists)
    lists[0, 0, 100:] = -1  # whole parts of the list without a block
    check_attend(s, lists)
    # as many tokens as fill the card without cutting, but parts longer than a CTA may hold
    s = Cache(kind, 8, 8, 64, [64 * 40] * 40, [1] * 40, 0, 64)
    lists = np.tile(np.arange(1500, dtype=np.int32) % 40, (40, 8, 1))
    out, st = run_attend(s, lists)
    at = [0, 39]
    c = dict(s.c, cached=[64 * 40] * 2, new=[1, 1], base=s.c["base"][at])
    want, tol = rb.attend(c, s.q64()[at], lists[at], s.entries("k"), s.entries("v"), kind != "bf16")
    assert st == 0 and (np.abs(out[at] - want) <= tol).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("keep", [3, 40])
def test_lists_that_leave_no_key_give_zeros(kind, keep):
    s = Cache(kind, 8, 2, 128, [3000, 10], [1, 2], 64, 64)
    lists = random_lists(s, keep, forms=False)
    lists[0, 1] = -1
    lists[2, 0] = 99
    out, st = run_attend(s, lists)
    assert st == 0 and (out[0, 4:] == 0).all() and (out[2, :4] == 0).all()
    check_attend(s, lists)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("block", [64, 256])
def test_entries_outside_the_lists_have_no_part(kind, block):
    """NaN and infinities in blocks that are not listed, behind the query and in other requests."""
    s = Cache(kind, 8, 2, 64, [700, 900], [3, 1], 256, block)
    lists = random_lists(s, 2, forms=False)
    lists[:, :, 1] = np.array([(700 + j) // block for j in range(3)] + [900 // block])[:, None]
    lists[:, :, 0] = 0
    want, tol = rb.attend(s.c, s.q64(), lists, s.entries("k"), s.entries("v"), kind != "bf16")
    listed = np.zeros(s.c["slots"], bool)
    t = 0
    for b, (c, n) in enumerate(zip(s.c["cached"], s.c["new"])):
        for i in {0, c // block, (c + n - 1) // block}:
            p = np.arange(i * block, min((i + 1) * block, c + n))
            listed[rb.slots_of(s.c, b, p)] = True
    bad = torch.tensor(~listed).cuda()
    for x, scales in ((s.kv.k_cache, s.kv.k_block_scale), (s.kv.v_cache, s.kv.v_block_scale)):
        if kind == "bf16":
            x[bad] = float("nan")
            x[bad.nonzero()[::2, 0]] = float("inf")
        elif kind == "e4m3":
            x[bad] = 0x7F
        else:
            scales[:, bad] = 0x7F
    out, st = run_attend(s, lists)
    assert st == 0 and (np.abs(out - want) <= tol).all()


@pytest.mark.parametrize("kind", KINDS)
def test_listed_entries_that_are_not_finite_show(kind):
    s = Cache(kind, 4, 2, 64, [500], [1], 64, 64)
    lists = random_lists(s, 3, forms=False)
    p = int(lists[0, 1, 1]) * 64 + 5
    slot = int(rb.slots_of(s.c, 0, [p])[0])
    if kind == "bf16":
        s.kv.v_cache[slot, 1, 0] = float("nan")
    elif kind == "e4m3":
        s.kv.v_cache[slot, 1, 0] = 0x7F
    else:
        s.kv.v_block_scale[1, slot, 0] = 0x7F
    out, _ = run_attend(s, lists)
    assert np.isnan(out[0, 2:, 0]).all() and np.isfinite(out[0, :2]).all()


@pytest.mark.parametrize("kind", KINDS)
def test_attend_problems_set_the_status(kind):
    s = Cache(kind, 4, 2, 64, [300, 400, 500], [2, 1, 2], 64, 64)
    lists = random_lists(s, 4, forms=False)
    # a page outside the cache reads as zeros
    page = int(lists[0, 0, 0])
    s.kv.page_table[0, page] = 1 << 20
    s.c["table"][0, page] = 1 << 20
    out, st = run_attend(s, lists)
    want, tol = rb.attend(s.c, s.q64(), lists, s.entries("k"), s.entries("v"), kind != "bf16")
    assert st == CAP and (np.abs(out - want) <= tol).all()
    # a region that is too small is skipped, and so are tokens behind the last request
    s.kv.slot_capacity[1] = 400
    out, st = run_attend(s, lists)
    assert st == CAP and (out[2] == 776).all() and (np.abs(out - want) <= tol)[[0, 1, 3, 4]].all()
    s.cu[3] = 4
    out, st = run_attend(s, lists)
    assert st & SEQ and (out[4] == 776).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page,block,extra", [(128, 128, 100), (256, 64, 130), (256, 256, 1)])
def test_a_page_that_the_cache_s_end_cuts(kind, page, block, extra):
    """Its number lies outside the cache: it has no bounds, scores as zeros and reads as zeros."""
    from causal_gqa_attention_qkv_gb300 import attn
    s = Cache(kind, 4, 2, 64, [page * 9 + 3], [page], page, block, extra_slots=extra)
    cut = s.c["slots"] // page
    for i in (2, 8):
        s.kv.page_table[0, i] = cut
        s.c["table"][0, i] = cut
    ws = s.workspace(4)
    attn.block_bounds(s.cfg, s.kv, s.blocks, s.cu, ws, start=i32([0]))
    assert status(ws) == CAP
    got, want = s.bounds.double().cpu().numpy(), rb.bounds(s.c, s.entries("k"), [0])
    for row in range(s.c["rows"]):
        assert np.array_equal(got[row], want.get(row, np.full_like(got[row], 776.0)))
    fill_bounds(s)
    lists, st = run_select(s, 1, 1, 4)
    assert st == CAP and np.array_equal(lists, rb.select(s.c, s.q64(), s.bounds.double().cpu().numpy(), 1, 1, 4))
    lists[:, :, 1] = 2 * page // block
    out, st = run_attend(s, lists)
    want, tol = rb.attend(s.c, s.q64(), lists, s.entries("k"), s.entries("v"), kind != "bf16")
    assert st == CAP and (np.abs(out - want) <= tol).all()


@pytest.mark.parametrize("kind", KINDS)
def test_attend_in_a_cache_past_two_to_the_32_bytes(kind):
    from causal_gqa_attention_qkv_gb300 import attn
    hkv, d, ps = 8, 128, 64
    row = hkv * {"bf16": 2 * d, "e4m3": d, "e2m1": d // 2}[kind]
    pages = (5 << 30) // row // ps
    s = Cache(kind, 8, hkv, d, [64 * 20 + 7], [1], ps, ps)
    lists = random_lists(s, 6, forms=False)
    want, tol = rb.attend(s.c, s.q64(), lists, s.entries("k"), s.entries("v"), kind != "bf16")
    old, n = s.kv, s.kv.k_cache.shape[0]
    first = pages * ps - n
    big = []
    for x in (old.k_cache, old.v_cache):
        y = torch.zeros(pages * ps, *x.shape[1:], dtype=x.dtype, device="cuda")
        y[first:] = x
        big.append(y)
    scales = []
    for x in (old.k_block_scale, old.v_block_scale):
        if x is not None:
            y = torch.zeros(hkv, pages * ps, d // 16, dtype=torch.uint8, device="cuda")
            y[:, first:] = x
            scales.append(y)
    s.kv = attn.KVCache(*big, old.slot_base, old.cache_lens, old.slot_capacity, old.page_table + first // ps, ps,
                        rb.K_SCALE, rb.V_SCALE, *scales)
    out, st = run_attend(s, lists)
    assert st == 0 and (np.abs(out - want) <= tol).all()


def test_attend_over_all_blocks_is_the_dense_call():
    from causal_gqa_attention_qkv_gb300 import attn
    s = Cache("bf16", 8, 2, 128, [700, 0, 64], [33, 130, 1], 64, 64)
    n = -(-max(c + m for c, m in zip(s.c["cached"], s.c["new"])) // 64)
    lists = np.tile(np.arange(n, dtype=np.int32), (s.N, s.hkv, 1))
    out, _ = run_attend(s, lists)
    dense = torch.empty(s.N, s.hq * s.d, dtype=torch.bfloat16, device="cuda")
    ws = attn.new_workspace(s.cfg, s.N, 3, 1024)
    attn.prefill_attend(s.cfg, s.q, s.cu, max(s.c["new"]), s.kv, dense, ws)
    # both round P (the dense call to bf16, 2^-8 of sum p |v|) and the output (2^-8)
    assert np.abs(out.reshape(s.N, -1) - dense.double().cpu().numpy()).max() <= 2.0 ** -5


# ------------------------------------------------------------------ refusals of the bindings
def test_bindings_refuse_what_does_not_fit():
    from causal_gqa_attention_qkv_gb300 import attn
    s = Cache("bf16", 4, 2, 64, [300, 400], [1, 1], 64, 64)
    ws, lists = s.workspace(4), i32(np.zeros((2, 2, 4)))
    out = torch.empty(2, 256, dtype=torch.bfloat16, device="cuda")
    sel = lambda **k: attn.block_select(**{**dict(cfg=s.cfg, q=s.q, cu_seqlens=None, max_kv_len=500, kv=s.kv,
                                                  blocks=s.blocks, first=1, last=1, out_list=lists, workspace=ws), **k})
    att = lambda **k: attn.block_attend(**{**dict(cfg=s.cfg, q=s.q, cu_seqlens=None, kv=s.kv, block_size=64,
                                                  block_list=lists, out=out, workspace=ws), **k})
    sel()
    att()
    for f in (sel, att):
        for bad in (dict(q=s.q.half()), dict(q=s.q[:1]), dict(q=s.q[:, :2]), dict(cu_seqlens=i32([0, 1, 2, 2])),
                    dict(cfg=attn.config(8, 4, 64)), dict(cu_seqlens=torch.tensor([0, 1, 2]).cuda())):
            with pytest.raises((AssertionError, attn.AttnError)):
                f(**bad)
    for f, bad in ((sel, dict(out_list=lists[:1])), (sel, dict(out_list=lists.long())), (sel, dict(first=4)),
                   (sel, dict(blocks=attn.BlockBounds(s.bounds.float(), 64))), (sel, dict(workspace=ws[:256])),
                   (sel, dict(blocks=attn.BlockBounds(s.bounds[:2], 64))), (att, dict(out=out[:1])),
                   (att, dict(block_list=lists[:, :1])), (att, dict(block_size=128)), (att, dict(block_size=63))):
        with pytest.raises((AssertionError, attn.AttnError)):
            f(**bad)
    with pytest.raises(AssertionError):
        attn.block_bounds(s.cfg, s.kv, s.blocks, None, ws, start=i32([0]))
    with pytest.raises(attn.AttnError):
        attn.new_block_workspace(s.cfg, 4, 100, 96, 4)


# ------------------------------------------------------------------ together
class Layer:
    """One layer's paged cache that grows: prepare, bounds, select, attend."""

    def __init__(self, kind, rows=6, pages=80, ppr=24, hq=8, hkv=2, d=64, page=128, block=64, keep=6):
        from causal_gqa_attention_qkv_gb300 import attn
        self.a = attn
        self.kind, self.block, self.keep, self.page = kind, block, keep, page
        self.cfg = attn.config(hq, hkv, d)
        w = {"bf16": d, "e4m3": d, "e2m1": d // 2}[kind]
        t = torch.bfloat16 if kind == "bf16" else torch.uint8
        k, v = (torch.zeros(pages * page, hkv, w, dtype=t, device="cuda") for _ in range(2))
        sc = [torch.zeros(hkv, pages * page, d // 16, dtype=torch.uint8, device="cuda") for _ in range(2)] if kind == "e2m1" \
            else [None, None]
        self.kv = attn.KVCache(k, v, torch.zeros(rows, dtype=torch.int64, device="cuda"), i32([0] * rows),
                               i32([ppr * page] * rows), torch.full((rows, ppr), -1, dtype=torch.int32, device="cuda"),
                               page, rb.K_SCALE, rb.V_SCALE, *sc)
        self.ref = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.pws = attn.new_pages_workspace(self.kv)
        self.blocks = attn.new_block_bounds(self.cfg, self.kv, block)
        self.ws = attn.new_block_workspace(self.cfg, 1000, ppr * page, block, keep)
        g = torch.Generator().manual_seed(3)
        self.qw, self.kw = ((1 + 0.1 * torch.randn(d, generator=g)).bfloat16().cuda() for _ in range(2))
        self.max_len = ppr * page

    def qkv(self, n, seed):
        c = self.cfg
        return torch.randn(n, (c.num_q_heads + 2 * c.num_kv_heads) * c.head_dim,
                           generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()

    def buffers(self, n):
        c = self.cfg
        q = torch.empty(n, c.num_q_heads, c.head_dim, device="cuda",
                        dtype=torch.bfloat16 if self.kind == "bf16" else torch.float16)
        lists = torch.empty(n, c.num_kv_heads, self.keep, dtype=torch.int32, device="cuda")
        return q, lists, torch.empty(n, c.num_q_heads * c.head_dim, dtype=torch.bfloat16, device="cuda")

    def step(self, qkv, cu, kv, q, lists, out, single=False, stream=None):
        a = self.a
        q_in = q if self.kind == "bf16" else q.view(torch.bfloat16)  # prefill_prepare's binding takes 16-bit words as bf16
        a.prefill_prepare(self.cfg, qkv, self.qw, self.kw, cu, kv, q_in, self.ws, stream=stream)
        c = None if single else cu
        a.block_bounds(self.cfg, kv, self.blocks, c, self.ws, stream=stream)
        a.block_select(self.cfg, q, c, self.max_len, kv, self.blocks, 1, 2, lists, self.ws, stream=stream)
        a.block_attend(self.cfg, q, c, kv, self.block, lists, out, self.ws, stream=stream)

    def check(self, cu, kv, q, lists, out):
        """What a step left against the plain forms, each from what the calls before it gave."""
        import ref64
        cached, new = kv.cache_lens.tolist(), np.diff(cu.cpu().numpy()).tolist()
        c = {"block": self.block, "page": self.page, "cached": cached, "new": new, "table": kv.page_table.cpu().numpy(),
             "slots": kv.k_cache.shape[0], "rows": self.blocks.bounds.shape[0], "row_base": None}
        scale = lambda s: 1.0 if self.kind == "bf16" else s
        keys = ref64.entries(kv.k_cache, self.kind, scale(rb.K_SCALE), kv.k_block_scale)
        vals = ref64.entries(kv.v_cache, self.kind, scale(rb.V_SCALE), kv.v_block_scale)
        bounds = self.blocks.bounds.double().cpu().numpy()
        for row, v in rb.bounds(c, keys, start=[0] * len(cached)).items():
            assert np.array_equal(bounds[row], v)
        x = q.double().cpu().numpy()
        want = rb.select(c, x, bounds, 1, 2, self.keep)
        assert np.array_equal(lists.cpu().numpy(), want)
        o, tol = rb.attend(c, x, want, keys, vals, self.kind != "bf16")
        assert (np.abs(out.double().cpu().numpy().reshape(o.shape) - o) <= tol).all()
        assert status(self.ws) == 0


@pytest.mark.parametrize("kind", KINDS)
def test_a_served_batch(kind):
    """Prompts in chunks, forks, single tokens, a moved pool: every step's bounds, lists and
    outputs against the plain forms over what the cache then holds."""
    y = Layer(kind)
    a = y.a
    rows = i32([0, 1, 2])
    a.pages_reserve(y.kv, y.ref, rows, i32([900, 130, 500]), y.pws)
    done = torch.zeros(3, dtype=torch.int32, device="cuda")
    for k, new in enumerate(([300, 100, 0], [400, 29, 450], [120, 0, 10])):
        cu = i32(np.concatenate(([0], np.cumsum(new))))
        kv = y.kv.rows(0, 3, done.clone())
        b = y.buffers(sum(new))
        y.step(y.qkv(sum(new), k), cu, kv, *b)
        y.check(cu, kv, *b)
        done += i32(new)
    y.kv.cache_lens[:3] = done
    # the first prompt is sampled twice: its open page is copied, and the full blocks of the copy get bounds
    a.pages_fork(y.cfg, y.kv, y.ref, i32([0, 0]), i32([3, 4]), y.pws)
    five = y.kv.rows(0, 5)
    start = (five.cache_lens // y.page * y.page).contiguous()
    a.block_bounds(y.cfg, five, y.blocks, i32([0] * 6), y.ws, start=start)
    cu = i32(range(6))
    for k in range(3):
        a.pages_reserve(y.kv, y.ref, i32(range(5)), i32([1] * 5), y.pws)
        kv = y.kv.rows(0, 5)
        b = y.buffers(5)
        y.step(y.qkv(5, 10 + k), cu, kv, *b, single=True)
        y.check(cu, kv, *b)
        y.kv.cache_lens[:5] += 1
    # a request ends, the pool is packed, the bounds of what moved are made anew
    a.pages_free(y.kv, y.ref, i32([1]), y.pws)
    a.pages_compact(y.cfg, y.kv, y.ref, y.pws)
    kv = y.kv.rows(0, 5)
    a.block_bounds(y.cfg, kv, y.blocks, i32([0] * 6), y.ws, start=i32([0] * 5))
    a.pages_reserve(y.kv, y.ref, i32([0, 2, 3, 4]), i32([1] * 4), y.pws)
    a.pages_reserve(y.kv, y.ref, i32([1]), i32([1]), y.pws)
    kv = y.kv.rows(0, 5)
    b = y.buffers(5)
    y.step(y.qkv(5, 20), cu, kv, *b, single=True)
    y.check(cu, kv, *b)
    assert a.get_status(y.pws) == 0


@pytest.mark.parametrize("kind", ["bf16", "e2m1"])
def test_captured_steps_replay(kind):
    """A captured step of single tokens, replayed as the cached lengths advance on the device."""
    y = Layer(kind)
    a = y.a
    a.pages_reserve(y.kv, y.ref, i32([0, 1, 2]), i32([1500, 700, 1100]), y.pws)
    cu0, new = i32([0, 400, 463, 500]), [400, 63, 37]
    kv = y.kv.rows(0, 3, i32([0, 0, 0]))
    b = y.buffers(500)
    y.step(y.qkv(500, 0), cu0, kv, *b)
    kv = y.kv.rows(0, 3, i32(new))
    cu, b = i32(range(4)), y.buffers(3)
    qkv = y.qkv(3, 1)
    eager, lens = [], kv.cache_lens
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y.step(qkv, cu, kv, *b, single=True)  # warm-up of the captured calls
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y.step(qkv, cu, kv, *b, single=True)
        lens += 1
    for k in range(5):
        qkv.copy_(y.qkv(3, 30 + k))
        for t in b[1:]:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        lens -= 1
        y.check(cu, kv, *b)
        lens += 1
    assert a.get_status(y.ws) == 0


def test_calls_on_another_stream_and_two_workspaces():
    """Two streams with a workspace each give what one gives."""
    s = [Cache("bf16", 8, 2, 64, [3000 + i, 5000], [1, 1], 64, 64, seed=i) for i in range(2)]
    want = []
    for x in s:
        fill_bounds(x)
        want.append(run_select(x, 1, 2, 9)[0])
    from causal_gqa_attention_qkv_gb300 import attn
    streams = [torch.cuda.Stream() for _ in s]
    ws = [x.workspace(9) for x in s]
    lists = [torch.zeros(2, 2, 9, dtype=torch.int32, device="cuda") for _ in s]
    outs = [torch.zeros(2, 512, dtype=torch.bfloat16, device="cuda") for _ in s]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, st, w, l, o in zip(s, streams, ws, lists, outs):
            attn.block_select(x.cfg, x.q, None, x.max_len, x.kv, x.blocks, 1, 2, l, w, stream=st)
            attn.block_attend(x.cfg, x.q, None, x.kv, 64, l, o, w, stream=st)
    torch.cuda.synchronize()
    for x, l, o, n in zip(s, lists, outs, want):
        assert np.array_equal(l.cpu().numpy(), n)
        ref, tol = rb.attend(x.c, x.q64(), n, x.entries("k"), x.entries("v"), False)
        assert (np.abs(o.double().cpu().numpy().reshape(ref.shape) - ref) <= tol).all()


def test_results_repeat_bit_for_bit():
    for kind in KINDS:
        s = Cache(kind, 8, 2, 128, [9000, 400, 64 * 100], [1, 1, 1], 64, 64)
        fill_bounds(s)
        lists, _ = run_select(s, 1, 2, 30)
        a, _ = run_attend(s, lists)
        for _ in range(3):
            again, _ = run_select(s, 1, 2, 30)
            assert np.array_equal(again, lists)
            b, _ = run_attend(s, lists)
            assert np.array_equal(a, b)
