"""GPU tests of the calls on logits (include/logits.h): every rule and their order
against the plain fp32 steps, bit for bit, at the sizes, alignments and lists where
they can go wrong; the table of seen tokens; and a decoding loop with the sampler."""
import numpy as np
import pytest
import torch

import ref_blocks as rb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_gqa_attention_qkv_gb300 import build
    build.build()


def dev(x, t):
    return torch.tensor(np.asarray(x), dtype=t).cuda()


class Rows:
    """B rows of logits with rules: seen tokens (a share `seen` of the vocabulary), biases
    (`biases` per row, `dup` of them again), masks that allow a share `mask`."""

    def __init__(self, B, V, seed=0, seen=0.05, biases=0, dup=0, mask=None, table_rows=None, shuffle=True):
        rng = np.random.RandomState(seed)
        self.B, self.V = B, V
        self.x = (3 * rng.randn(B, V)).astype(np.float32)
        R = table_rows or B + 2
        self.seen = None
        if seen is not None:
            w = np.where(rng.rand(R, V) < seen, rng.randint(0, 6, (R, V)) | (rng.randint(0, 2, (R, V)) << 15), 0)
            w[:, rng.randint(V, size=3)] = 0x7FFF
            self.seen = np.zeros((R, -(-V // 8) * 8), np.int16)
            self.seen[:, :V] = np.where(w >= 0x8000, w - 0x10000, w)
            self.seen[:, V:] = 5  # words behind the vocabulary have no part
        self.row = rng.permutation(R)[:B] if shuffle else np.arange(B)
        self.rep = (1 + rng.rand(B)).astype(np.float32)
        self.pres, self.freq = (rng.randn(2, B) * 0.5).astype(np.float32)
        self.bias = []
        for b in range(B):
            t = rng.randint(0, V, biases)
            t = np.concatenate((t, rng.choice(t, dup) if biases else t)).astype(int)
            rng.shuffle(t)
            self.bias.append([(int(v), np.float32(rng.randn())) for v in t])
        self.mask = None
        if mask is not None:
            self.mask = rng.rand(max(1, B // 2), V) < mask
            self.mask_row = rng.randint(-1, self.mask.shape[0], B)

    def rules(self, **change):
        from causal_gqa_attention_qkv_gb300 import attn
        f = {}
        if self.seen is not None:
            f.update(seen=dev(self.seen, torch.int16), seen_row=dev(self.row, torch.int32),
                     repetition=dev(self.rep, torch.float32), presence=dev(self.pres, torch.float32),
                     frequency=dev(self.freq, torch.float32))
        if any(self.bias):
            f.update(bias_start=dev(np.cumsum([0] + [len(x) for x in self.bias]), torch.int32),
                     bias_token=dev([t for x in self.bias for t, _ in x], torch.int32),
                     bias_value=dev([v for x in self.bias for _, v in x], torch.float32))
        if self.mask is not None:
            words = -(-self.V // 32)
            bits = np.zeros((self.mask.shape[0], words * 32), np.uint32)
            bits[:, :self.V] = self.mask
            bits[:, self.V:] = 1  # bits behind the vocabulary have no part
            m = (bits.reshape(-1, words, 32) << np.arange(32, dtype=np.uint32)).sum(-1, dtype=np.uint32)
            f.update(mask=dev(m.view(np.int32), torch.int32), mask_row=dev(self.mask_row, torch.int32))
        f.update(change)
        return attn.LogitsRules(**f)

    def want(self, rep=True, pres=True, freq=True):
        out = []
        for b in range(self.B):
            r = self.row[b]
            s = None
            if self.seen is not None and 0 <= r < self.seen.shape[0]:
                s = self.seen[r, :self.V]
            m = None
            if self.mask is not None and 0 <= self.mask_row[b] < self.mask.shape[0]:
                m = self.mask[self.mask_row[b]]
            out.append(rb.adjust(self.x[b], s, self.rep[b] if rep else None, self.pres[b] if pres else None,
                                 self.freq[b] if freq else None, self.bias[b], m))
        return np.stack(out)


def run(x, rules, out=None):
    from causal_gqa_attention_qkv_gb300 import attn
    return attn.logits_adjust(x, rules, out=out).cpu().numpy()


def check(w, rules=None, **kw):
    x = dev(w.x, torch.float32)
    got = run(x, rules or w.rules(), torch.full_like(x, 99.0))
    assert np.array_equal(got, w.want(**kw), equal_nan=True)
    assert np.array_equal(x.cpu().numpy(), w.x, equal_nan=True)


@pytest.mark.parametrize("B,V", [(1, 1), (1, 7), (3, 33), (2, 511), (2, 512), (2, 513), (5, 1023), (1, 1025), (3, 4099),
                                 (1, 151936), (64, 32000), (7, 32003), (700, 1030)])
@pytest.mark.parametrize("biases,mask", [(0, None), (9, 0.3)])
def test_every_rule(B, V, biases, mask):
    check(Rows(B, V, seed=V, biases=biases, dup=biases // 3, mask=mask))


@pytest.mark.parametrize("name", ["seen", "repetition", "presence", "frequency", "bias_start", "mask"])
def test_rules_left_out(name):
    w = Rows(3, 3001, biases=20, mask=0.5)
    r = w.rules(**{name: None})
    if name == "seen":
        w.seen = None
    if name == "bias_start":
        w.bias = [[]] * 3
    if name == "mask":
        w.mask = None
    check(w, r, rep=name != "repetition", pres=name != "presence", freq=name != "frequency")
    from causal_gqa_attention_qkv_gb300 import attn
    w.seen, w.bias, w.mask = None, [[]] * 3, None
    check(w, attn.LogitsRules())


@pytest.mark.parametrize("seen", [0.0, 0.5, 1.0])
def test_few_and_many_seen_tokens(seen):
    check(Rows(4, 5000, seen=seen, biases=3, mask=0.5))
    check(Rows(2, 300, seen=seen))


@pytest.mark.parametrize("V,biases,dup", [(100, 100, 100), (700, 127, 0), (700, 129, 1), (2000, 3000, 500), (1024, 128, 0),
                                          (40000, 20000, 0)])
def test_many_biases(V, biases, dup):
    """Around the number that a run handles one per thread, and far past it."""
    check(Rows(3, V, seed=biases, biases=biases, dup=dup))


def test_one_token_biased_again_and_again():
    w = Rows(2, 900)
    rng = np.random.RandomState(0)
    w.bias = [[(5, np.float32(rng.randn() * 10 ** rng.randint(-3, 4))) for _ in range(120)], []]
    check(w)
    w.bias = [[], [(899, np.float32(rng.randn() * 10 ** rng.randint(-3, 4))) for _ in range(5000)]]
    check(w)


def test_tokens_and_rows_outside():
    w = Rows(4, 1000, biases=10, mask=0.5)
    w.bias[1] += [(-1, np.float32(3)), (1000, np.float32(3)), (2 ** 31 - 1, np.float32(3)), (-2 ** 31, np.float32(3))]
    w.row = np.array([-1, 10 ** 6, w.seen.shape[0], 0])
    w.mask_row = np.array([5, -7, 0, 10 ** 8])
    check(w)


def test_biases_named_outside_the_list():
    """bias_start that begins before the list, ends past it or runs backwards."""
    w = Rows(4, 1500, biases=9)
    r = w.rules()
    r.bias_start = dev([-5, 18, 30, 27, 10 ** 9], torch.int32)
    w.bias = [w.bias[0] + w.bias[1], w.bias[2] + w.bias[3][:3], [], w.bias[3]]
    check(w, r)
    r.bias_start = dev([40, 2 ** 31 - 1, -2 ** 31, -1, 0], torch.int32)
    w.bias = [[]] * 4
    check(w, r)


def test_rows_by_their_own_number():
    """No row numbers: row b of the table and of the masks."""
    w = Rows(3, 777, mask=0.4, shuffle=False, table_rows=3)
    w.mask = np.random.RandomState(1).rand(3, 777) < 0.4
    w.mask_row = np.arange(3)
    check(w, w.rules(seen_row=None, mask_row=None))
    # fewer rows than logits: the others have none
    w = Rows(3, 777, shuffle=False, table_rows=3)
    r = w.rules(seen_row=None)
    r.seen = r.seen[:2].contiguous()
    w.seen = w.seen[:2]
    check(w, r)


@pytest.mark.parametrize("offset,ld,ld_out,off_out", [(0, 1003, 1003, 0), (1, 1001, 1004, 0), (4, 1004, 1001, 3), (0, 1004, 1008, 4),
                                                      (2, 1000, 1000, 2), (3, 1002, 1002, 3)])
def test_rows_that_start_anywhere(offset, ld, ld_out, off_out):
    """Strided rows and storage offsets; what lies between the rows stays."""
    w = Rows(5, 1000, biases=12, mask=0.5)
    store = torch.full((5 * ld + 8,), 7.0, device="cuda")
    x = store[offset:].as_strided((5, 1000), (ld, 1))
    x.copy_(dev(w.x, torch.float32))
    dst = torch.full((5 * ld_out + 8,), 55.0, device="cuda")
    out = dst[off_out:].as_strided((5, 1000), (ld_out, 1))
    assert np.array_equal(run(x, w.rules(), out), w.want())
    out.fill_(55.0)
    assert (dst == 55).all()
    # in place
    from causal_gqa_attention_qkv_gb300 import attn
    assert attn.logits_adjust(x, w.rules()) is x
    assert np.array_equal(x.cpu().numpy(), w.want())
    x.fill_(7.0)
    assert (store == 7).all()


@pytest.mark.parametrize("V,biases", [(151936, 300), (3000, 2000), (33, 40), (5000, 0)])
def test_in_place(V, biases):
    w = Rows(4, V, biases=biases, dup=biases // 4, mask=0.2)
    x = dev(w.x, torch.float32)
    assert np.array_equal(run(x, w.rules()), w.want())


def test_logits_that_are_not_finite():
    w = Rows(2, 640, seen=0.6, biases=60, dup=20, mask=0.7)
    rng = np.random.RandomState(5)
    w.x[rng.rand(2, 640) < 0.2] = -np.inf
    w.x[rng.rand(2, 640) < 0.1] = np.inf
    w.x[rng.rand(2, 640) < 0.1] = np.nan
    w.x[rng.rand(2, 640) < 0.1] = -0.0
    w.x[rng.rand(2, 640) < 0.1] = 1e-42
    w.bias[0][:6] = [(t, np.float32(v)) for (t, _), v in zip(w.bias[0], [np.inf, -np.inf, np.nan, 3e38, 3e38, -1e-44])]
    for rep in ([0.0, -1.0], [np.nan, np.inf], [1e-40, 1e38], [1.0, 0.5]):
        w.rep = np.array(rep, np.float32)
        check(w)
    w.freq, w.pres = np.array([np.inf, -np.inf], np.float32), np.array([np.nan, 1e38], np.float32)
    check(w)


@pytest.mark.parametrize("V,biases", [(1000, 0), (1000, 100), (500, 128), (500, 129), (1000, 300), (5000, 3000)])
def test_zeros_keep_their_sign(V, biases):
    """Bit for bit, -0 among them: a logit without a bias does not depend on how many of its
    neighbours have one (a run's biases are summed in another way from 129 on)."""
    w = Rows(3, V, seed=biases, seen=0.2, biases=biases, dup=biases // 10, mask=0.7)
    w.x[np.random.RandomState(7).rand(3, V) < 0.6] = -0.0
    w.bias = [[(t, np.float32(-0.0) if t % 3 == 0 else v) for t, v in x] for x in w.bias]
    for x, out in ((dev(w.x, torch.float32), None), (dev(w.x, torch.float32), torch.empty(3, V, device="cuda"))):
        got, want = run(x, w.rules(), out), w.want()
        assert np.signbit(want).any() and np.array_equal(got.view(np.int32), want.view(np.int32))


def test_masks_that_allow_nothing():
    w = Rows(3, 2000, biases=5, mask=0.0)
    w.mask_row[:] = 0
    got = run(dev(w.x, torch.float32), w.rules())
    assert (got == -np.inf).all()


def test_no_rows():
    from causal_gqa_attention_qkv_gb300 import attn
    x = torch.empty(0, 100, device="cuda")
    assert attn.logits_adjust(x, attn.LogitsRules()).shape == (0, 100)
    seen = attn.new_seen(2, 100)
    attn.tokens_seen(seen, 100, dev([], torch.int32), dev([], torch.int32))
    attn.tokens_seen(seen, 100, dev([0, 1], torch.int32), dev([], torch.int32), dev([0, 0, 0], torch.int32))
    assert (seen == 0).all()


# ------------------------------------------------------------------ seen tokens
def check_seen(table, vocab, rows, groups, **kw):
    from causal_gqa_attention_qkv_gb300 import attn
    t = dev(table, torch.int16)
    cu = np.cumsum([0] + [len(g) for g in groups])
    attn.tokens_seen(t, vocab, dev(rows, torch.int32), dev([v for g in groups for v in g], torch.int32),
                     dev(cu, torch.int32), **kw)
    want = rb.seen_rows(table, vocab, rows, groups, **kw)
    assert np.array_equal(t.cpu().numpy(), want)
    return want


@pytest.mark.parametrize("prompt", [False, True])
@pytest.mark.parametrize("clear", [False, True])
@pytest.mark.parametrize("vocab", [1, 9, 8192, 8193, 32003, 151936])
def test_seen(prompt, clear, vocab):
    rng = np.random.RandomState(vocab)
    table = np.where(rng.rand(6, -(-vocab // 8) * 8 + 8) < 0.1, rng.randint(-32768, 32768, (6, -(-vocab // 8) * 8 + 8)), 0)
    groups = [rng.randint(-2, vocab + 2, n).tolist() for n in (0, 1, 700, 33, 5000)]
    check_seen(table.astype(np.int16), vocab, [4, 0, 5, 2, 1], groups, prompt=prompt, clear=clear)


@pytest.mark.parametrize("prompt", [False, True])
@pytest.mark.parametrize("clear", [False, True])
def test_rows_named_again_and_rows_outside(prompt, clear):
    rng = np.random.RandomState(1)
    rows = [3, -1, 3, 0, 99, 3, 0] + [2] * 400
    groups = [rng.randint(0, 50, rng.randint(9)).tolist() for _ in rows]
    check_seen(np.full((4, 64), 7, np.int16), 50, rows, groups, prompt=prompt, clear=clear)


def test_counts_stop_at_their_largest():
    for clear in (False, True):
        check_seen(np.full((2, 16), 32700, np.int16), 16, [1], [[3] * 70000 + [4] * 50 + [5] * 67], clear=clear)
    table = np.full((1, 8), -32768 + 32766, np.int16)  # in the prompt, 32766 times
    assert check_seen(table, 8, [0], [[1, 1, 2]])[0, :3].tolist() == [-2, -1, -1]


def test_single_tokens_and_rows_by_their_own_number():
    from causal_gqa_attention_qkv_gb300 import attn
    rng = np.random.RandomState(2)
    for B in (1, 31, 300, 5000):
        t = attn.new_seen(B, 100)
        tok = rng.randint(0, 100, B)
        attn.tokens_seen(t, 100, None, dev(tok, torch.int32))
        attn.tokens_seen(t, 100, None, dev(tok, torch.int32))
        attn.tokens_seen(t, 100, None, dev(tok[::-1].copy(), torch.int32), prompt=True)
        want = rb.seen_rows(np.zeros((B, 104), np.int16), 100, range(B), [[v, v] for v in tok])
        want = rb.seen_rows(want, 100, range(B), [[v] for v in tok[::-1]], prompt=True)
        assert np.array_equal(t.cpu().numpy(), want)


def test_a_table_past_two_to_the_32_bytes():
    from causal_gqa_attention_qkv_gb300 import attn
    vocab, rows = 151936, 15000
    seen = attn.new_seen(rows, vocab)
    last = rows - 1
    attn.tokens_seen(seen, vocab, dev([last, last - 1], torch.int32), dev([5, 151935, 7], torch.int32),
                     dev([0, 2, 3], torch.int32), clear=True)
    attn.tokens_seen(seen, vocab, dev([last], torch.int32), dev([5], torch.int32))
    assert seen[last].nonzero()[:, 0].tolist() == [5, 151935] and seen[last, 5] == 2 and seen[last - 1, 7] == 1
    assert not seen[:1000].any()
    x = torch.ones(1, vocab, device="cuda")
    attn.logits_adjust(x, attn.LogitsRules(seen=seen, seen_row=dev([last], torch.int32),
                                           frequency=torch.ones(1, device="cuda")))
    assert x[0, 5] == -1 and x[0, 151935] == 0 and x[0, 7] == 1


@pytest.mark.parametrize("prompt", [False, True])
def test_rows_of_more_than_two_to_the_31_words(prompt):
    """Emptied whole, each segment in its place, and nothing before them."""
    from causal_gqa_attention_qkv_gb300 import attn
    ld = (1 << 31) + 3 * 8192 + 16
    seen = torch.full((2, ld), 5, dtype=torch.int16, device="cuda")
    attn.tokens_seen(seen, 9000, dev([1], torch.int32), dev([7, 8999, 7, 9000, -1], torch.int32), dev([0, 5], torch.int32),
                     prompt=prompt, clear=True)
    assert seen[1, 7] == (-32768 if prompt else 2) and seen[1, 8999] == (-32768 if prompt else 1)
    seen[1, 7] = seen[1, 8999] = 0
    for row, value in ((0, 5), (1, 0)):
        for part in seen[row].split(1 << 28):
            assert (part == value).all()


# ------------------------------------------------------------------ refusals of the bindings
def test_bindings_refuse_what_does_not_fit():
    from causal_gqa_attention_qkv_gb300 import attn
    w = Rows(3, 500, biases=4, mask=0.5)
    x, r = dev(w.x, torch.float32), w.rules()
    run(x, r)
    for bad in (x.half(), x.cpu(), x.t(), x[0]):
        with pytest.raises(AssertionError):
            attn.logits_adjust(bad, r)
    with pytest.raises(AssertionError):
        attn.logits_adjust(x, r, out=x[:2])
    for name, t in (("seen_row", r.seen_row[:2]), ("seen_row", r.seen_row.long()), ("repetition", r.repetition.double()),
                    ("bias_start", r.bias_start[:3]), ("bias_value", r.bias_value[:2]), ("bias_token", None),
                    ("mask", r.mask.long()), ("mask", r.mask[:, ::2]), ("mask_row", r.mask_row[:1]), ("seen", r.seen.int()),
                    ("seen", r.seen[0])):
        with pytest.raises((AssertionError, attn.AttnError)):
            attn.logits_adjust(x, w.rules(**{name: t}))
    with pytest.raises(attn.AttnError):
        attn.logits_adjust(x, w.rules(mask=r.mask[:, :15].contiguous()))
    with pytest.raises(attn.AttnError):
        attn.logits_adjust(x, w.rules(seen=r.seen[:, :496].contiguous()))
    with pytest.raises(AssertionError):
        attn.logits_adjust(x[:2], r)
    seen, tok = attn.new_seen(3, 500), dev([1, 2, 3], torch.int32)
    for kw in (dict(seen=seen.int()), dict(rows=dev([0, 1], torch.int32)), dict(tokens=tok.long()), dict(vocab=505),
               dict(cu_seqlens=dev([0, 3], torch.int64)), dict(vocab=0)):
        with pytest.raises((AssertionError, attn.AttnError)):
            attn.tokens_seen(**{**dict(seen=seen, vocab=500, rows=None, tokens=tok), **kw})


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("captured", [False, True])
def test_a_decoding_loop(captured):
    """Prompts marked, then steps of adjust, sample, count: the table and every row of logits
    against the plain forms, and no token that a mask forbids or that a penalty buries."""
    from causal_gqa_attention_qkv_gb300 import attn
    B, V, steps = 5, 4001, 6
    rng = np.random.RandomState(3)
    w = Rows(B, V, biases=7, mask=0.3, table_rows=9)
    w.mask_row = np.array([-1, 0, 1, 0, -1])
    w.freq[:] = 100.0  # no token twice
    seen = attn.new_seen(9, V)
    r = w.rules(seen=seen)
    prompts = [rng.randint(0, V, n).tolist() for n in (3, 900, 1, 50, 20)]
    attn.tokens_seen(seen, V, r.seen_row, dev([t for p in prompts for t in p], torch.int32),
                     dev(np.cumsum([0] + [len(p) for p in prompts]), torch.int32), prompt=True, clear=True)
    table = rb.seen_rows(np.zeros((9, seen.shape[1]), np.int16), V, w.row, prompts, prompt=True)
    x = torch.empty(B, V, device="cuda")
    y, u = torch.empty_like(x), torch.empty(B, device="cuda")
    tokens = torch.empty(B, dtype=torch.int32, device="cuda")
    temp, top_k, top_p = torch.tensor([0.0, 1.0, 0.7, 2.0, 1.0]).cuda(), dev([0, 5, 0, 50, 0], torch.int32), \
        torch.tensor([1.0, 1.0, 0.9, 1.0, 1.0]).cuda()

    def step():
        attn.logits_adjust(x, r, out=y)
        attn.sample_tokens(y, temp, top_k, top_p, u, tokens)
        attn.tokens_seen(seen, V, r.seen_row, tokens)
    graph = None
    if captured:
        x.zero_()
        u.fill_(0.5)
        before = seen.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        seen.copy_(before)
    drawn = []
    for k in range(steps):
        w.x = (3 * rng.randn(B, V)).astype(np.float32)
        x.copy_(dev(w.x, torch.float32))
        u.copy_(dev(rng.rand(B), torch.float32))
        w.seen = table
        want = w.want()
        graph.replay() if captured else step()
        assert np.array_equal(y.cpu().numpy(), want)
        t = tokens.cpu().numpy()
        assert np.isfinite(want[np.arange(B), t]).all() and t[0] == want[0].argmax()
        drawn.append(t)
        table = rb.seen_rows(table, V, w.row, [[v] for v in t])
        assert np.array_equal(seen.cpu().numpy(), table)
    for b in range(B):
        assert len({int(t[b]) for t in drawn}) == steps
