"""The cache's operators together, as a server uses them: a prompt with an image (three axes) is written, two users go on
from it (fork), each drafts a tree; its attention, the verification, the compaction of the kept path and the pages given
back.  After every step the cache holds what one would hold that had written the settled tokens alone."""
import pytest
import torch

import _cacheref as R

pytestmark = pytest.mark.gpu
I32 = torch.int32
HEADS, GROUP, DIM, PAGE, VOCAB = 2, 2, 64, 16, 90


@pytest.fixture(scope="module")
def mx():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from microscaling_quantize_dequantize_amd import binding
    return binding


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


class Server:
    def __init__(self, mx, fmt, pages=64, seed=0):
        self.mx, self.g = mx, torch.Generator().manual_seed(seed)
        self.cache = mx.MXCache.allocate(fmt, pages, HEADS, PAGE, DIM)
        self.refs = torch.zeros(pages, dtype=I32, device="cuda")
        pairs = DIM // 2
        self.inv_freq = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device="cuda") / pairs)
        self.axes = i32([p % 3 for p in range(pairs)])
        self.weights = torch.randn((VOCAB, HEADS * (GROUP + 2), DIM), generator=self.g).bfloat16().cuda()
        self.logits = 2.0 * torch.randn((VOCAB, VOCAB), generator=self.g)

    def new(self, tokens, positions, table, lens):
        """Writes tokens (a list for each row of the table) behind lens, with pages for them."""
        counts = [len(t) for t in tokens]
        missing = self.mx.mx_cache_resize(self.cache, self.refs, table, i32([n + c for n, c in zip(lens, counts)]))
        assert not bool(missing.any())
        slots = [int(table[b, p // PAGE]) * PAGE + p % PAGE for b, n in enumerate(lens) for p in range(n, n + counts[b])]
        qkv = self.weights[torch.tensor([t for row in tokens for t in row], device="cuda")]
        q, k, v = qkv[:, :HEADS * GROUP], qkv[:, HEADS * GROUP:-HEADS], qkv[:, -HEADS:]
        at = torch.tensor(positions, device="cuda").T.contiguous()
        self.mx.mx_cache_write(self.cache, k, v, torch.tensor(slots, device="cuda"), positions=at, inv_freq=self.inv_freq,
                               axes=self.axes)
        return self.mx.mx_rope(q, at, self.inv_freq, axes=self.axes)

    def tokens_of(self, table, b, n):
        p = torch.arange(n, device="cuda")
        return self.mx.mx_cache_read(self.cache, table[b].long()[p // PAGE] * PAGE + p % PAGE)


def text(n):
    return [n, n, n]


@pytest.mark.parametrize("fmt", [0, 1])
def test_a_server(mx, fmt):
    s = Server(mx, fmt, seed=fmt)
    rnd = lambda *shape: torch.rand(shape, generator=s.g, dtype=torch.float64)  # noqa: E731
    # a prompt: 10 of text, 24 of an image (4 rows of 6 at one time), 5 of text behind it
    prompt = torch.randint(0, VOCAB, (39,), generator=s.g).tolist()
    positions = [text(i) for i in range(10)] + [[10, 10 + i // 6, 10 + i % 6] for i in range(24)] + \
        [text(16 + i) for i in range(5)]
    table = torch.full((1, 6), -1, dtype=I32, device="cuda")
    s.new([prompt], positions, table, [0])
    assert s.refs.tolist().count(1) == 3
    # the image's tokens alone, in the first two pages and a part of the third: text of another length looks at them
    q = s.weights[torch.randint(0, VOCAB, (7,), generator=s.g), :HEADS * GROUP].contiguous()
    starts, lens = i32([0, 7]), i32([34])
    seen = mx.mx_cache_cross_attention(s.cache, q, starts, lens, table, max_q=7, max_kv=34)
    for i in range(7):  # each is what a single new token would see
        one = mx.mx_cache_attention(s.cache, q[i:i + 1], i32([0, 1]), lens, table, max_q=1, max_kv=34)
        ref, weight, size = R.attention(s.cache, q[i:i + 1], i32([0, 1]), lens, table)
        bound = R.attention_bound(ref, weight + ref.abs(), size, DIM, 34)
        for got in (seen[i:i + 1], one):
            assert bool(((got.double().cpu() - ref).abs() <= bound).all())
    # two users go on from it; the pages that are full are shared
    table, missing = mx.mx_cache_fork(s.cache, s.refs, table, i32([39]), i32([0, 0]))
    assert missing.tolist() == [0, 0] and s.refs[table[0, :2].long()].tolist() == [3, 3]
    assert table[0, :2].tolist() == table[1, :2].tolist() and table[0, 2] != table[1, 2]
    settled = [list(prompt), list(prompt)]
    where = [list(positions), list(positions)]
    last = [prompt[-1], prompt[-1]]  # to be written with its drafts
    n = [38, 38]
    sizes = [7, 12]
    for step in range(4):
        # drafted trees: node 0 is the last settled token, which is at n[b]
        parents = [[-1] + [int(rnd(1) * min(i, 4)) + max(0, i - 4) for i in range(1, m)] for m in sizes]
        p = torch.softmax(s.logits, 1)
        drafts, depth, rows = [], [], []
        for b, m in enumerate(sizes):
            tok, dep, q_rows = [last[b]], [0], []
            for i in range(1, m):
                up = parents[b][i]
                q = torch.softmax(s.logits[tok[up]] + 0.5 * torch.sin(torch.arange(VOCAB) * 1.3), 0)
                c = q.double().cumsum(0)
                tok.append(min(int(torch.searchsorted(c, rnd(1) * c[-1], right=True)), VOCAB - 1))
                dep.append(dep[up] + 1)
            for t in tok:
                q_rows.append(torch.softmax(s.logits[t] + 0.5 * torch.sin(torch.arange(VOCAB) * 1.3), 0))
            drafts.append(tok)
            depth.append(dep)
            rows += q_rows
        at = [text(where[b][n[b] - 1][0] + 1 + d) if step or d else where[b][n[b]] for b in range(2) for d in depth[b]]
        q = s.new(drafts, at, table, n)
        words = []
        for b, m in enumerate(sizes):
            bits = [1]
            for i in range(1, m):
                bits.append(bits[parents[b][i]] | (1 << i))
            words += bits
        starts = i32([0, sizes[0], sum(sizes)])
        kv = i32([x + m for x, m in zip(n, sizes)])
        tree = torch.tensor(words, device="cuda")[:, None]
        out = mx.mx_cache_attention(s.cache, q, starts, kv, table, max_q=max(sizes), max_kv=80, tree=tree)
        ref, weight, size = R.attention(s.cache, q, starts, kv, table, tree)
        assert bool(((out.double().cpu() - ref).abs() <= R.attention_bound(ref, weight + ref.abs(), size, DIM, 60)).all())
        target = p[torch.tensor([t for row in drafts for t in row])].cuda()
        tokens = torch.tensor([t for row in drafts for t in row], device="cuda")
        counts, path, put = mx.mx_verify(target, tokens, rnd(sum(sizes)).cuda(), starts, max(sizes),
                                         draft=torch.stack(rows).cuda(), parents=i32(parents[0] + parents[1]))
        before = [s.tokens_of(table, b, n[b] + sizes[b]) for b in range(2)]
        after = mx.mx_cache_compact(s.cache, i32(n), path, counts, table)
        missing = mx.mx_cache_resize(s.cache, s.refs, table, after)
        assert not bool(missing.any()) and after.tolist() == [x + int(c) for x, c in zip(n, counts)]
        for b in range(2):
            kept = path[b, :int(counts[b])].tolist()
            assert put[b, :len(kept) - 1].tolist() == [drafts[b][i] for i in kept[1:]]
            assert all(parents[b][j] == i for i, j in zip(kept, kept[1:]))
            k, v = s.tokens_of(table, b, n[b] + len(kept))
            rows_kept = list(range(n[b])) + [n[b] + i for i in kept]
            assert torch.equal(k, before[b][0][rows_kept]) and torch.equal(v, before[b][1][rows_kept])
            first = sum(sizes[:b])
            where[b] = where[b][:n[b]] + [at[first + i] for i in kept]
            settled[b] = settled[b][:n[b]] + [drafts[b][i] for i in kept]
            last[b] = int(put[b, len(kept) - 1])
            assert 0 <= last[b] < VOCAB
            n[b] += len(kept)
    # what is there now is what writing the settled tokens in one go gives
    fresh = Server(mx, fmt, seed=fmt)
    for b in range(2):
        alone = torch.full((1, 8), -1, dtype=I32, device="cuda")
        fresh.new([settled[b]], where[b], alone, [0])
        for x, y in zip(s.tokens_of(table, b, n[b]), fresh.tokens_of(alone, 0, n[b])):
            assert torch.equal(x, y)
    # the users leave; the prompt's own row still holds its three pages
    mx.mx_cache_resize(s.cache, s.refs, table, i32([0, 0]))
    assert sorted(s.refs.tolist())[-3:] == [1, 1, 1] and int(s.refs.sum()) == 3
