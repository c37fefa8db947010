"""Attention over the paged MX cache against softmax in 64 bits, with a bound
derived from the roundings: formats, head sizes and groups, one token to many,
pages that end inside a unit, ragged and empty sequences, trees, rows that see
nothing, NaN and bad pages, splits, strides, streams, graphs, far offsets."""
import pytest
import torch

import _cacheref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from microscaling_quantize_dequantize_amd import binding
    return binding


class Case:
    """Sequences of kv tokens (the new ones among them) with random codes in shuffled pages."""

    def __init__(self, mx, fmt, heads, group, dim, page, kv, nq, seed=0, spread=1.0, spare=2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g = g
        need = [-(-n // page) for n in kv]
        pages = sum(need) + spare
        self.cache = mx.MXCache.allocate(fmt, pages, heads, page, dim)
        c = self.cache
        for t in (c.k_codes, c.v_codes):
            t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
            if fmt == 1:
                t[(t & 127) == 127] = 1  # no NaN codes
        for t in (c.k_scales, c.v_scales):
            low = 124 if fmt == 0 else 116
            t.copy_(torch.randint(low, low + 4, t.shape, generator=g, device="cuda", dtype=torch.uint8))
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((len(kv), max(max(need), 1)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.kv, self.nq = kv, nq
        self.kv_lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
        self.q_starts = torch.tensor([sum(nq[:i]) for i in range(len(nq) + 1)], dtype=torch.int32, device="cuda")
        self.q = (spread * torch.randn((sum(nq), heads * group + 1, dim), generator=g, device="cuda")).bfloat16()[:, 1:]
        self.tree = None

    def random_tree(self):
        words = -(-max(self.nq) // 64)
        rows = []
        for n in self.nq:
            for i in range(n):
                see = (torch.rand(n, generator=self.g, device="cuda") < 0.4).tolist()
                see[i] = True
                row = [0] * words
                for j, s in enumerate(see):
                    if s:
                        row[j // 64] |= 1 << (j % 64)
                rows.append([w - (1 << 64) if w >> 63 else w for w in row])
        self.tree = torch.tensor(rows, dtype=torch.int64, device="cuda").reshape(sum(self.nq), words)
        return self

    def run(self, mx, **kw):
        return mx.mx_cache_attention(self.cache, self.q, self.q_starts, self.kv_lens, self.table, max_q=max(self.nq),
                                     max_kv=max(self.kv), tree=self.tree, **kw)

    def check(self, out, scale=None):
        ref, weight, size = R.attention(self.cache, self.q, self.q_starts, self.kv_lens, self.table, self.tree, scale)
        got = out.double().cpu()
        bound = R.attention_bound(ref, weight, size, ref.shape[2], max(self.kv))
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        over = torch.where(torch.isnan(ref), 0.0, (got - ref).abs() - bound)
        assert float(over.max()) <= 0, (float(over.max()), float((got - ref).abs().nan_to_num().max()))


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("group,nq", [(1, 1), (4, 1), (8, 3), (5, 12), (3, 45)])
def test_heads_and_rows(mx, fmt, dim, group, nq):
    """From one row of a key/value head to more than a workgroup's."""
    c = Case(mx, fmt, 2, group, dim, 16, [nq + 70, nq], [nq, max(1, nq // 2)], seed=dim + nq)
    c.check(c.run(mx))


@pytest.mark.parametrize("fmt,dim", [(0, 64), (1, 128), (1, 192)])
@pytest.mark.parametrize("group", [16, 17, 71])
def test_one_key_value_head_for_many(mx, fmt, dim, group):
    """A single token whose query heads alone are more rows than a block of the few-rows kernel."""
    c = Case(mx, fmt, 1, group, dim, 32, [700, 33], [1, 1], seed=group)
    c.check(c.run(mx))


@pytest.mark.parametrize("page", [16, 32, 64, 256])
@pytest.mark.parametrize("kv", [1, 2, 15, 16, 17, 63, 64, 65, 255, 256, 257, 1000])
def test_lengths_and_pages(mx, page, kv):
    c = Case(mx, 1, 2, 4, 128, page, [kv], [1], seed=kv)
    c.check(c.run(mx))


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dim,group", [(64, 7), (128, 4), (256, 2)])
def test_splits(mx, fmt, dim, group):
    """Sequences over several workgroups' spans, ragged, one of them short, one empty, one without queries."""
    c = Case(mx, fmt, 1, group, dim, 32, [5000, 1, 0, 300, 2600], [1, 1, 1, 0, 2], seed=dim)
    c.check(c.run(mx))


@pytest.mark.parametrize("group,nq", [(2, 1), (4, 10)])
def test_many_sequences(mx, group, nq):
    """More sequences than a wave has lanes, most of them short, some without tokens or queries: the division of the
    work passes over them."""
    kv = [(37 * b) % 91 for b in range(150)]
    kv[3], kv[77], kv[149] = 1500, 900, 700
    new = [0 if b % 11 == 5 else 1 + b % nq for b in range(150)]
    c = Case(mx, 1, 1, group, 64, 16, kv, new, seed=150)
    c.check(c.run(mx))


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("nodes,kv", [(2, 2), (13, 400), (16, 16), (64, 300), (65, 65), (100, 731), (130, 700)])
def test_trees(mx, fmt, nodes, kv):
    c = Case(mx, fmt, 2, 2, 64, 16, [kv, nodes + 3], [nodes, max(1, nodes - 1)], seed=nodes).random_tree()
    c.check(c.run(mx))


@pytest.mark.parametrize("chunk,kv", [(40, 40), (100, 1000), (333, 700)])
def test_chunks_of_a_prompt(mx, chunk, kv):
    c = Case(mx, 1, 1, 4, 128, 64, [kv, chunk // 2 + 1], [chunk, chunk // 3], seed=chunk)
    c.check(c.run(mx))


def test_rows_that_see_nothing_are_zero(mx):
    """Empty tree rows without a prefix; more queries than tokens; a sequence of no tokens."""
    c = Case(mx, 1, 2, 2, 64, 16, [20, 5, 0], [20, 9, 3], seed=4).random_tree()
    c.tree[3] = 0
    c.tree[19] = 0
    out = c.run(mx)
    c.check(out)
    assert not bool(out[3].any()) and not bool(out[19].any()) and not bool(out[29:].any())
    c.tree = None  # causal: the first four of nine queries over five tokens see none
    out = c.run(mx)
    c.check(out)
    assert not bool(out[20:24].any()) and bool(out[24].any())


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("tree", [False, True])
def test_nan_reaches_only_rows_that_see_it(mx, fmt, tree):
    """NaN keys and values among the new tokens, and garbage behind the sequence's end in its last page."""
    nq, kv = 20, 90
    c = Case(mx, fmt, 1, 2, 128, 16, [kv], [nq], seed=11)
    if tree:
        c.random_tree()
    pages = c.table[0].tolist()

    def scale_byte(t, tok, group):
        t[pages[tok // 16], 0, group, tok % 16] = 255

    scale_byte(c.cache.v_scales, kv - 4, 1)   # a value of new token 16
    scale_byte(c.cache.k_scales, kv - 7, 2)   # a key of new token 13
    for tok in range(kv, 96):                 # behind the end
        for grp in range(4):
            scale_byte(c.cache.v_scales, tok, grp)
            scale_byte(c.cache.k_scales, tok, grp)
    out = c.run(mx)
    c.check(out)
    assert bool(torch.isnan(out).any()) and not bool(torch.isnan(out[:13]).all())


@pytest.mark.parametrize("group,nq", [(2, 4), (4, 20), (8, 20)])
def test_nan_in_some_of_many_sequences(mx, group, nq):
    """Items that need their NaN next to items that do not, several to a workgroup and divided over several."""
    kv = [700 + 13 * b for b in range(12)]
    c = Case(mx, 1, 2, group, 64, 16, kv, [nq] * 12, seed=31).random_tree()
    for b in range(0, 12, 3):
        for tok in (kv[b] - 2, kv[b] - nq):
            c.cache.v_codes[int(c.table[b, tok // 16]), 1, tok % 16, 7] = 0x7F
    out = c.run(mx)
    c.check(out)
    assert bool(torch.isnan(out).any())


@pytest.mark.parametrize("bad", [-1, 1 << 30, -(1 << 31)])
def test_pages_outside_the_cache_are_not_seen(mx, bad):
    c = Case(mx, 1, 2, 4, 64, 32, [700, 64], [3, 1], seed=2)
    c.table[0, 2] = bad
    c.table[0, 21] = bad  # the last page
    c.table[1, 0] = bad
    c.check(c.run(mx))
    c.table[1, 1] = bad   # all of the second sequence
    out = c.run(mx)
    c.check(out)
    assert not bool(out[3].any())


@pytest.mark.parametrize("spread", [1e-3, 30.0])
def test_flat_and_peaked_scores(mx, spread):
    c = Case(mx, 1, 2, 4, 128, 64, [900], [2], seed=8, spread=spread)
    c.check(c.run(mx))
    c.check(c.run(mx, scale=0.011), scale=0.011)


def test_rising_scores_rescale(mx):
    """Scores that grow along the sequence by more than the maximum may lag."""
    c = Case(mx, 1, 1, 1, 64, 64, [2000], [1], seed=3)
    ramp = 100 + torch.arange(2000) * 27 // 2000
    t = torch.arange(2000)
    pages = c.table[0].cpu()[t // 64].long()
    c.cache.k_scales[pages.cuda(), 0, 0, (t % 64).cuda()] = ramp.to(torch.uint8).cuda()
    c.cache.k_scales[pages.cuda(), 0, 1, (t % 64).cuda()] = ramp.to(torch.uint8).cuda()
    c.check(c.run(mx))


def test_max_lengths_may_be_larger(mx):
    c = Case(mx, 0, 2, 2, 96, 16, [100, 40], [2, 1], seed=6)
    want = c.run(mx)
    got = mx.mx_cache_attention(c.cache, c.q, c.q_starts, c.kv_lens, c.table, max_q=50, max_kv=100000)
    c.check(want)
    c.check(got)


def test_offsets_past_32_bits(mx):
    """The last pages of a cache of more than 2^32 bytes of codes."""
    heads, page, dim = 16, 256, 128
    pages = (1 << 32) // (heads * page * dim) + 3
    cache = mx.MXCache.allocate(1, pages, heads, page, dim)
    c = Case(mx, 1, heads, 1, dim, page, [600], [1], seed=7, spare=0)
    old = c.table[0].long()
    new = torch.tensor([pages - 1, 2, pages - 3], device="cuda")
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        getattr(cache, n)[new] = getattr(c.cache, n)[old]
    want = c.run(mx)
    c.cache, c.table = cache, new.to(torch.int32)[None]
    assert torch.equal(c.run(mx), want)


def test_results_repeat_and_other_streams(mx):
    c = Case(mx, 1, 2, 4, 128, 64, [6000, 3000], [1, 1], seed=12)
    want = c.run(mx)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = [c.run(mx) for _ in range(3)]
    s.synchronize()
    for o in got:
        assert torch.equal(o, want)


def test_captured_step_replays_like_eager(mx):
    """Rotate the queries, write, attend, read back in one graph; replayed with eager work in between."""
    heads, group, dim, page = 2, 4, 128, 64
    c = Case(mx, 1, heads, group, dim, page, [3000, 500], [1, 1], seed=13)
    slots = torch.tensor([int(c.table[0, 2999 // page]) * page + 2999 % page,
                          int(c.table[1, 499 // page]) * page + 499 % page], device="cuda")
    pos = torch.tensor([2999, 499], device="cuda")
    f = 10000.0 ** (-torch.arange(dim // 2, dtype=torch.float64, device="cuda") / (dim // 2))
    q = c.q.contiguous()
    k, v = (torch.randn((2, heads, dim), device="cuda").bfloat16() for _ in range(2))
    out, qr = torch.empty_like(q), torch.empty_like(q)
    rk, rv = torch.empty_like(k), torch.empty_like(k)

    def step():
        mx.mx_rope(q, pos, f, dst=qr)
        mx.mx_cache_write(c.cache, k, v, slots, positions=pos, inv_freq=f)
        mx.mx_cache_attention(c.cache, qr, c.q_starts, c.kv_lens, c.table, max_q=1, max_kv=3000, out=out)
        mx.mx_cache_read(c.cache, slots, k=rk, v=rv)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rep in range(3):
        q.copy_(torch.randn_like(q))
        k.copy_(torch.randn_like(k))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (out, qr, rk, rv)]
        for t in (out, qr, rk, rv):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for t, w in zip((out, qr, rk, rv), want):
            assert torch.equal(t, w), rep


def test_nothing_to_do(mx):
    cache = mx.MXCache.allocate(0, 1, 2, 16, 64)
    q = torch.empty((0, 4, 64), device="cuda").bfloat16()
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = mx.mx_cache_attention(cache, q, zero, zero[:2], torch.zeros((2, 1), dtype=torch.int32, device="cuda"), 0, 0)
    assert out.shape == (0, 4, 64)
