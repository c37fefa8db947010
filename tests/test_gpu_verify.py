"""mx_verify against exact rational arithmetic: chains and trees, with and without the drafts' probabilities, sizes that
end inside a load, strides and alignments, empty sequences and padding, probabilities that are no numbers, refusals that
leave nothing, and the distribution of what comes out."""
import math

import pytest
import torch

import _verifyref as V

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from microscaling_quantize_dequantize_amd import binding
    return binding


class Case:
    """Drafted nodes whose tokens are drawn from noisy copies of the target's probabilities."""

    def __init__(self, sizes, vocab, dtype=torch.float32, tree=False, draft=True, seed=0, noise=0.7, width=5, cut=True):
        g = torch.Generator().manual_seed(seed)
        total = sum(sizes)
        x = 2.0 * torch.randn((total, vocab), generator=g)
        y = x + noise * torch.randn((total, vocab), generator=g)
        p, q = torch.softmax(x, 1), torch.softmax(y, 1)
        if cut and vocab > 4:
            p, q = torch.where(p > 0.3 / vocab, p, 0.0), torch.where(q > 0.3 / vocab, q, 0.0)
            p, q = p / p.sum(1, keepdim=True), q / q.sum(1, keepdim=True)
        self.target, q = p.to(dtype).cuda(), q.to(dtype)
        node = torch.cat([torch.arange(n) for n in sizes])
        back = torch.rand(total, generator=g)
        parent = node - 1 - (back * node.clamp(max=width)).long() if tree else node - 1
        parent = parent.clamp(min=-1)
        first = torch.arange(total) - node
        c = q[first + parent.clamp(min=0)].double().cumsum(1)
        r = torch.rand((total, 1), generator=g, dtype=torch.float64) * c[:, -1:]
        self.tokens = torch.searchsorted(c, r, right=True)[:, 0].clamp(max=vocab - 1).cuda()
        self.parents = parent.to(torch.int32).cuda() if tree else None
        self.draft = q.cuda() if draft else None
        self.uniforms = torch.rand(total, generator=g, dtype=torch.float64).cuda()
        starts = [0]
        for n in sizes:
            starts.append(starts[-1] + n)
        self.q_starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
        self.max_q = max(sizes)

    def run(self, mx, **kw):
        f = dict(target=self.target, tokens=self.tokens, uniforms=self.uniforms, q_starts=self.q_starts,
                 max_q=self.max_q, draft=self.draft, parents=self.parents)
        return mx.mx_verify(**{**f, **kw})

    def check(self, got, max_q=None):
        want = V.verify(self.target, self.tokens, self.uniforms, self.q_starts, max_q or self.max_q, self.draft,
                        self.parents)
        for name, a, b in zip(("counts", "path", "tokens"), got, want):
            assert a.dtype == b.dtype and torch.equal(a.cpu(), b), (name, a.cpu(), b)
        return want


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("vocab", [1, 2, 3, 4, 5, 7, 8, 9, 31, 64, 65, 257, 1000])
def test_vocabularies(mx, dtype, tree, draft, vocab):
    c = Case([9, 1, 4, 6, 2], vocab, dtype, tree, draft, seed=vocab)
    c.check(c.run(mx))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("vocab", [8191, 8200, 33001])
def test_rows_over_several_workgroups(mx, dtype, draft, vocab):
    for tree in (False, True):
        c = Case([7, 5], vocab, dtype, tree, draft, seed=vocab)
        c.check(c.run(mx))


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("sizes,width", [([64, 17, 1, 40], 5), ([200], 60), ([1024, 3], 300), ([65, 64, 63], 64)])
def test_many_nodes(mx, draft, sizes, width):
    """Trees up to the most nodes, in which nodes have many children (and so many refusals)."""
    c = Case(sizes, 40, tree=True, draft=draft, seed=sum(sizes), width=width, noise=3.0)
    c.check(c.run(mx))


def test_a_long_chain(mx):
    """Every draft is kept: p and q are the same, which the test of a draft always passes."""
    c = Case([1024, 30], 50, seed=3, noise=0.0)
    counts, path, out = c.run(mx)
    assert counts.tolist() == [1024, 30]
    assert torch.equal(path[0].cpu(), torch.arange(1024, dtype=torch.int32))
    c.check((counts, path, out))


def test_many_sequences(mx):
    sizes = [(7 * b) % 11 for b in range(300)]
    for tree in (False, True):
        c = Case(sizes, 37, tree=tree, seed=8)
        c.check(c.run(mx))


@pytest.mark.parametrize("tree", [False, True])
def test_empty_and_bounded(mx, tree):
    """Sequences without nodes, a bound below the nodes of a sequence, rows behind the last sequence."""
    c = Case([0, 6, 0, 9, 3, 0], 33, tree=tree, seed=21)
    c.check(c.run(mx))
    for most in (1, 2, 5):
        c.check(c.run(mx, max_q=most), max_q=most)
    counts, path, out = c.run(mx, max_q=0)
    assert path.shape == out.shape == (6, 0) and counts.tolist() == [0] * 6
    c.q_starts = c.q_starts[:4].contiguous()  # the rest of the nodes belongs to nobody
    c.check(c.run(mx))
    none = c.run(mx, q_starts=c.q_starts[:1].contiguous())
    assert [tuple(t.shape) for t in none] == [(0,), (0, c.max_q), (0, c.max_q)]
    nothing = mx.mx_verify(c.target[:0], c.tokens[:0], c.uniforms[:0], torch.zeros(3, dtype=torch.int32, device="cuda"), 4)
    assert nothing[0].tolist() == [0, 0] and bool((nothing[1] == -1).all()) and bool((nothing[2] == -1).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("p_off,q_off,wide", [(0, 0, 64), (1, 1, 65), (3, 2, 71), (0, 5, 68), (7, 7, 80)])
def test_strides_and_alignments(mx, dtype, p_off, q_off, wide):
    """Rows inside wider ones, from any element on."""
    c = Case([6, 5, 9], 53, dtype, True, True, seed=p_off + wide)
    for name, off in (("target", p_off), ("draft", q_off)):
        t = getattr(c, name)
        big = torch.full((t.shape[0], wide), 9.0, dtype=dtype, device="cuda")  # not to be read as probabilities
        big[:, off:off + 53] = t
        setattr(c, name, big[:, off:off + 53])
    c.check(c.run(mx))
    shared = c.target[:1].expand(20, 53)  # one row for all nodes
    c.target = shared
    c.check(c.run(mx))


@pytest.mark.parametrize("draft", [False, True])
def test_nodes_that_are_passed_over(mx, draft):
    """Tokens outside the vocabulary, parents that are not before their nodes."""
    c = Case([12, 12, 12], 19, tree=True, draft=draft, seed=5)
    c.tokens[[2, 14, 17, 30]] = torch.tensor([-1, 19, 1 << 40, -(1 << 50)], device="cuda")
    c.parents[[4, 16, 19, 27, 35]] = torch.tensor([4, 9, -3, 1 << 30, -(1 << 31)], dtype=torch.int32, device="cuda")
    c.check(c.run(mx))
    c.parents = None
    want = c.check(c.run(mx))
    assert int(want[0][0]) <= 2  # a chain ends at such a token


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("draft", [False, True])
def test_probabilities_that_are_none(mx, dtype, draft):
    """NaN and negative entries count as zero, infinity as the largest number, in the walk and in the sample; a row of
    nothing gives -1."""
    c = Case([8, 8, 8, 8], 45, dtype, True, draft, seed=17)
    bad = torch.tensor([math.nan, math.inf, -math.inf, -0.25], dtype=dtype, device="cuda")
    for t in (c.target, c.draft):
        if t is not None:
            t[:, 3::11] = bad
    c.tokens[[1, 9, 18]] = torch.tensor([3, 14, 25], device="cuda")
    c.check(c.run(mx))
    c.target[16:24] = math.nan
    c.target[24:] = 0.0
    want = c.check(c.run(mx))
    assert want[2][2:, 0].tolist() == [-1, -1]


@pytest.mark.parametrize("vocab", [6, 300])
def test_refusals_that_leave_nothing(mx, vocab):
    """p below q everywhere, or on the drafted token alone: the weights stay as they were."""
    total = 4
    p = torch.zeros((total, vocab), device="cuda")
    p[:, 2], p[:, 4] = 0.25, 0.5
    q = torch.zeros((total, vocab), device="cuda")
    q[:, 2], q[:, 4] = 0.5, 0.5
    c = Case([4], vocab, tree=True, seed=1)
    c.target, c.draft = p, q
    c.tokens = torch.tensor([0, 2, 2, 4], device="cuda")
    c.parents = torch.tensor([-1, 0, 0, 0], dtype=torch.int32, device="cuda")
    for u in (0.0, 0.3, 0.6, 1.0 - 2.0 ** -53):
        c.uniforms = torch.tensor([u, 0.9, 0.75, 1.5], dtype=torch.float64, device="cuda")
        want = c.check(c.run(mx))
        assert want[2][0, 0] == (2 if u * 0.75 < 0.25 else 4)
    c.draft = None  # one token has it all, and is refused by a number that is none of [0, 1)
    c.target = torch.zeros((total, vocab), device="cuda")
    c.target[:, 4] = 1.0
    c.tokens[:] = 4
    c.uniforms = torch.tensor([0.5, 1.0, 1.0, 2.0], dtype=torch.float64, device="cuda")
    want = c.check(c.run(mx))
    assert want[2][0, 0] == 4


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_borders_of_the_sample(mx, dtype):
    """The first token whose cumulative sum is above u: entries without weight are never it, and the last one with
    weight is where u lets none be."""
    vocab = 5000
    p = torch.zeros((1, vocab), dtype=dtype, device="cuda")
    p[0, 17], p[0, 18], p[0, 3000], p[0, 4990] = 0.25, 0.25, 0.25, 0.25
    starts = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    token = torch.zeros(1, dtype=torch.int64, device="cuda")
    for u, want in ((0.0, 17), (0.25 - 2.0 ** -54, 17), (0.25, 18), (0.5, 3000), (0.75 - 2.0 ** -53, 3000), (0.75, 4990),
                    (1.0 - 2.0 ** -53, 4990), (1.0, 4990), (math.nan, 4990)):
        out = mx.mx_verify(p, token, torch.tensor([u], dtype=torch.float64, device="cuda"), starts, 1)[2]
        assert out.tolist() == [[want]], u


def test_large_vocabulary_against_64_bits(mx):
    """200003 entries: the walk in exact arithmetic would take long, so p and q differ in the first nodes alone and the
    sample goes by torch's 64-bit sums.  Sums in another order differ by some 1e-13 of the total at most, and the
    nearest border to a goal here is further off, which is asserted."""
    vocab = 200003
    for dtype, draft in ((torch.float32, True), (torch.bfloat16, False), (torch.bfloat16, True)):
        c = Case([3, 2, 5, 4], vocab, dtype, False, draft, seed=4)
        counts, path, out = (t.cpu() for t in c.run(mx))
        for b, at in enumerate([0, 3, 5, 10]):
            n = [3, 2, 5, 4][b]
            k = 0
            for i in range(1, n):
                x = int(c.tokens[at + i])
                p = float(c.target[at + i - 1, x])
                q = float(c.draft[at + i - 1, x]) if draft else 1.0
                if not float(c.uniforms[at + i]) * q < p:
                    break
                assert int(out[b, k]) == x
                k += 1
            assert int(counts[b]) == k + 1
            w = c.target[at + k].double()
            if k + 1 < n:
                if draft:
                    w = (w - c.draft[at + k].double()).clamp(min=0)
                else:
                    w[int(c.tokens[at + k + 1])] = 0.0
            cum = w.cumsum(0)
            goal = float(c.uniforms[at]) * float(cum[-1])
            assert float((cum - goal).abs().min()) > 1e-12 * float(cum[-1])
            assert int(out[b, k]) == int((cum > goal).float().argmax())


@pytest.mark.parametrize("draft", [False, True])
def test_the_target_is_what_comes_out(mx, draft):
    """Drafted siblings (independent draws from q, or any tokens without one) change the first token's distribution by
    nothing: each of 6 tokens' counts in 2^18 runs is binomial, so within 6 deviations."""
    n, vocab, nodes = 1 << 18, 6, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    p = torch.tensor([0.5, 0.02, 0.2, 0.0, 0.18, 0.1], device="cuda")
    q = torch.tensor([0.1, 0.3, 0.2, 0.2, 0.1, 0.1], device="cuda")
    target, drafts = p.expand(n * nodes, vocab), q.expand(n * nodes, vocab)
    tokens = torch.multinomial(q, n * nodes, replacement=True, generator=g)
    parents = torch.tensor([-1, 0, 0, 0], dtype=torch.int32, device="cuda").repeat(n)
    starts = torch.arange(0, n * nodes + 1, nodes, dtype=torch.int32, device="cuda")
    u = torch.rand(n * nodes, generator=g, dtype=torch.float64, device="cuda")
    counts, path, out = mx.mx_verify(target, tokens, u, starts, nodes, draft=drafts if draft else None, parents=parents)
    assert int(counts.min()) == 1 and int(counts.max()) == 2
    seen = torch.bincount(out[:, 0], minlength=vocab).double()
    want = n * p.double() / p.double().sum()
    assert bool(((seen - want).abs() <= 6 * (want * (1 - p.double())).sqrt() + 1e-9).all()), seen / n
    # with the drafts' probabilities more of them are kept than any single one would be
    if draft:
        assert float((counts == 2).double().mean()) > float(torch.minimum(p, q).sum())


def test_streams_and_replays(mx):
    """A captured call on its own stream, replayed between eager ones, for new numbers each time."""
    c = Case([9, 30, 4], 4001, tree=True, seed=6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.run(mx)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = c.run(mx)
    other = Case([5, 5], 3000, seed=7)
    for k in range(4):
        c.uniforms.copy_(torch.rand(43, dtype=torch.float64, generator=torch.Generator().manual_seed(k)))
        graph.replay()
        other.check(other.run(mx))
        torch.cuda.synchronize()
        c.check(held)


def test_rows_behind_4_gib(mx):
    """Rows 2^31 elements apart: strides and offsets are of 64 bits."""
    c = Case([3], 500, torch.bfloat16, seed=2)
    far = 1 << 31
    for name in ("target", "draft"):
        big = torch.empty(2 * far + 1000, dtype=torch.bfloat16, device="cuda")
        rows = big.as_strided((3, 500), (far, 1), 3)
        rows.copy_(getattr(c, name))
        setattr(c, name, rows)
    got = c.run(mx)
    c.target, c.draft = c.target.clone(), c.draft.clone()
    c.check(got)


def test_two_streams_at_once(mx):
    """Every call has a workspace of its own."""
    cases = [Case([30] * 6, 40001, torch.bfloat16, True, True, seed=k) for k in range(2)]
    want = [c.run(mx) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for k, c in enumerate(cases):
            with torch.cuda.stream(streams[k]):
                got[k].append(c.run(mx))
    torch.cuda.synchronize()
    for k in range(2):
        for g in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[k]))


def test_results_repeat(mx):
    c = Case([40] * 8, 50001, torch.bfloat16, True, True, seed=12)
    first = c.run(mx)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(c.run(mx), first))
