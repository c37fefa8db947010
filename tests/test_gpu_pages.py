"""The cache's pages against plain Python on lists and host tensors: copies, forks, taking and freeing, compaction; sizes
from one entry to more than a workgroup's step, pools that run out, tables with holes and bad numbers, strides, replays."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu
NAMES = ("k_codes", "k_scales", "v_codes", "v_scales")
I32 = torch.int32


@pytest.fixture(scope="module")
def mx():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from microscaling_quantize_dequantize_amd import binding
    return binding


def cache_of(mx, fmt, pages, heads, page, dim, seed=0):
    """A cache of random bytes: nothing here computes with them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    cache = mx.MXCache.allocate(fmt, pages, heads, page, dim)
    for n in NAMES:
        t = getattr(cache, n)
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    return cache


def snapshot(cache):
    return {n: getattr(cache, n).cpu().clone() for n in NAMES}


def same(cache, want):
    for n in NAMES:
        assert torch.equal(getattr(cache, n).cpu(), want[n]), n


def token(t, name, page, row):
    """A token's bytes of one tensor, all heads."""
    return t[page, :, row] if name.endswith("codes") else t[page, :, :, row]


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def grid(table):
    return i32(table).reshape(len(table), len(table[0]) if table else 0)


# ---- plain forms ---------------------------------------------------------------


def resize(refs, table, lens, page):
    """On lists, in place; the pages that each row needs and did not get."""
    pages, cols = len(refs), len(table[0]) if table else 0
    need = [-(-max(n, 0) // page) for n in lens]
    for r, row in enumerate(table):
        for j, p in enumerate(row):
            held = 0 <= p < pages
            if j >= need[r]:
                if held and refs[p] > 0:
                    refs[p] -= 1
                row[j] = -1
            elif not held:
                row[j] = -1
    free = iter([p for p in range(pages) if refs[p] == 0])
    missing = [max(0, n - cols) for n in need]
    for r, row in enumerate(table):
        for j in range(min(need[r], cols)):
            if row[j] == -1:
                p = next(free, None)
                if p is None:
                    missing[r] += 1
                else:
                    row[j] = p
                    refs[p] = 1
    return missing


def fork(refs, table, lens, parents, page, data=None):
    pages, cols = len(refs), len(table[0]) if table else 0
    children, missing, copies = [], [], []
    for s in parents:
        n = max(lens[s], 0) if 0 <= s < len(lens) else 0
        row = [-1] * cols
        for j in range(min(n // page, cols)):
            if 0 <= table[s][j] < pages:
                row[j] = table[s][j]
                refs[row[j]] += 1
        children.append(row)
        missing.append(max(0, -(-n // page) - cols))
    free = iter([p for p in range(pages) if refs[p] == 0])
    for c, s in enumerate(parents):
        n = max(lens[s], 0) if 0 <= s < len(lens) else 0
        j = n // page
        if n % page and j < cols:
            p = next(free, None)
            if p is not None:
                children[c][j] = p
                refs[p] = 1
                copies.append((table[s][j], p, n % page))
        missing[c] += sum(children[c][k] == -1 for k in range(min(-(-n // page), cols)))
    if data is not None:
        for src, dst, rows in copies:
            for name in NAMES:
                if 0 <= src < pages:
                    for r in range(rows):
                        token(data[name], name, dst, r).copy_(token(data[name], name, src, r))
    return children, missing


def compact(data, starts, keep, counts, table, page, pages):
    """All reads before all writes, by sequence."""
    cols = len(table[0]) if table else 0
    lens = []
    for b, start in enumerate(starts):
        count = max(min(counts[b], len(keep[b])), 0)
        lens.append(start + count)

        def at(place):
            if not 0 <= place < cols * page or not 0 <= table[b][place // page] < pages:
                return None
            return table[b][place // page], place % page

        moves = [(at(start + keep[b][i]), at(start + i)) for i in range(count) if keep[b][i] >= i]
        moves = [(s, d) for s, d in moves if s is not None and d is not None]
        for name in NAMES:
            old = [token(data[name], name, *s).clone() for s, _ in moves]
            for (_, d), bytes_ in zip(moves, old):
                token(data[name], name, *d).copy_(bytes_)
    return lens


# ---- copy ------------------------------------------------------------------------


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("heads,page,dim", [(1, 16, 32), (3, 16, 96), (2, 64, 128), (5, 32, 256), (1, 512, 64)])
def test_copy(mx, fmt, heads, page, dim):
    cache = cache_of(mx, fmt, 12, heads, page, dim)
    want = snapshot(cache)
    src, dst = [3, 0, 3, 7, -1, 12, 5, 1 << 30, 9], [1, 2, 4, 6, 8, 10, 99, 10, 9]
    for s, d in zip(src, dst):
        if 0 <= s < 12 and 0 <= d < 12:
            for n in NAMES:
                want[n][d] = want[n][s]
    mx.mx_cache_copy(cache, i32(src), i32(dst))
    same(cache, want)
    mx.mx_cache_copy(cache, i32([]), i32([]))
    same(cache, want)


def test_copy_many(mx):
    cache = cache_of(mx, 1, 6000, 2, 16, 64)
    want = snapshot(cache)
    order = torch.randperm(6000, generator=torch.Generator().manual_seed(3))
    src, dst = order[:3000], order[3000:]
    for n in NAMES:
        want[n][dst] = want[n][src]
    mx.mx_cache_copy(cache, src.to(I32).cuda(), dst.to(I32).cuda())
    same(cache, want)


# ---- taking and freeing -------------------------------------------------------------


def check_resize(mx, cache, refs, table, lens, stride=None):
    r, t = i32(refs), grid(table)
    if stride:
        wide = torch.full((t.shape[0], stride), 77, dtype=I32, device="cuda")
        wide[:, 1:1 + t.shape[1]] = t
        t = wide[:, 1:1 + t.shape[1]]
    got = mx.mx_cache_resize(cache, r, t, i32(lens))
    want = resize(refs, table, lens, cache.page)
    assert got.tolist() == want and t.tolist() == table and r.tolist() == refs
    if stride:
        assert bool((wide[:, 0] == 77).all()) and bool((wide[:, 1 + t.shape[1]:] == 77).all())


@pytest.mark.parametrize("rows,cols,pages,page", [(1, 1, 1, 16), (3, 5, 20, 16), (70, 9, 300, 32), (2, 700, 900, 16),
                                                  (40, 130, 9000, 64), (1500, 3, 20000, 16), (9, 1000, 8193, 16)])
def test_resize(mx, rows, cols, pages, page):
    """Rows that grow, shrink and end, call after call; some tables are wider than a step, some pools than a scan."""
    cache = mx.MXCache.allocate(0, pages, 1, page, 32)
    rng = random.Random(rows)
    refs, table = [0] * pages, [[-1] * cols for _ in range(rows)]
    for k in range(5):
        lens = [rng.choice([0, rng.randint(0, cols * page), rng.randint(0, page)]) for _ in range(rows)]
        check_resize(mx, cache, refs, table, lens, cols + 4 if k % 2 and rows > 1 else None)
    check_resize(mx, cache, refs, table, [0] * rows)
    assert refs == [0] * pages


def test_resize_without_enough(mx):
    """A pool that runs out gives what it has, in order; rows longer than the table say so; what is freed in a call is
    handed out in it."""
    cache = mx.MXCache.allocate(1, 10, 1, 16, 32)
    refs, table = [0] * 10, [[-1] * 4 for _ in range(4)]
    check_resize(mx, cache, refs, table, [64, 33, 64, 17])
    assert sum(r > 0 for r in refs) == 10
    check_resize(mx, cache, refs, table, [0, 33, 1000, 90])
    check_resize(mx, cache, refs, table, [64, -5, 1 << 30, 16])
    none = mx.MXCache.allocate(1, 0, 1, 16, 32)
    check_resize(mx, none, [], [[-1] * 3], [20])
    assert mx.mx_cache_resize(cache, i32(refs), i32([]).reshape(0, 4), i32([])).tolist() == []
    assert mx.mx_cache_resize(cache, i32(refs), i32([]).reshape(2, 0), i32([16, 17])).tolist() == [1, 2]


def test_resize_of_odd_tables(mx):
    """Holes, numbers outside the cache, a page twice, one that nobody is said to hold, reserved ones."""
    cache = mx.MXCache.allocate(0, 40, 1, 16, 32)
    refs = [0] * 40
    refs[0] = refs[1] = -1  # never handed out
    refs[7], refs[9], refs[3] = 2, 1, 5
    table = [[7, -1, 9, 40, -9, 3], [1 << 30, 7, 3, 12, 3, -1], [-1] * 6]
    check_resize(mx, cache, refs, table, [16 * 5, 16 * 1, 16 * 2 + 1])
    check_resize(mx, cache, refs, table, [16 * 1, 0, 16 * 6])
    check_resize(mx, cache, refs, table, [0, 0, 0])
    assert refs[:2] == [-1, -1] and refs[12] == 0


@pytest.mark.parametrize("rows,cols", [(60, 100), (1030, 7), (3, 5000)])
def test_resize_of_large_odd_tables(mx, rows, cols):
    """More entries than one workgroup sees to, with holes before held pages, and a pool whose low pages are taken."""
    pages, low = 90000, 70001
    cache = mx.MXCache.allocate(0, pages, 1, 16, 32)
    rng = random.Random(cols)
    refs = [1] * low + [0] * (pages - low)
    refs[40000] = refs[33] = 0
    table = [[-1] * cols for _ in range(rows)]
    check_resize(mx, cache, refs, table, [rng.randint(0, 16 * cols) for _ in range(rows)])
    for _ in range(3):  # holes; what is taken out is given back by hand
        for row in rng.sample(table, rows // 3 + 1):
            for j in rng.sample(range(cols), min(cols, 40)):
                if row[j] >= 0:
                    refs[row[j]] -= 1
                    row[j] = rng.choice([-1, -7, pages, 1 << 30])
        check_resize(mx, cache, refs, table, [rng.randint(0, 16 * cols) for _ in range(rows)])
    check_resize(mx, cache, refs, table, [16 * cols + 40] * rows)


# ---- forks ------------------------------------------------------------------------------


def check_fork(mx, cache, refs, table, lens, parents, out=None):
    data = snapshot(cache)
    r, t = i32(refs), grid(table)
    got, missing = mx.mx_cache_fork(cache, r, t, i32(lens), i32(parents), out=out)
    want, lack = fork(refs, table, lens, parents, cache.page, data)
    assert got.tolist() == want and missing.tolist() == lack and r.tolist() == refs and t.tolist() == table
    assert out is None or got is out
    same(cache, data)
    return want


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("heads,page,dim", [(1, 16, 32), (3, 16, 96), (2, 128, 64), (4, 32, 128)])
def test_fork(mx, fmt, heads, page, dim):
    """Children of some sequences, of none, of one that is not there; full last pages, one token, none."""
    pages = 40
    cache = cache_of(mx, fmt, pages, heads, page, dim)
    lens = [3 * page, 2 * page + 5, 1, 0, page - 1, page + 17 % page, 4 * page]
    refs, table = [0] * pages, [[-1] * 4 for _ in lens]
    resize(refs, table, lens, page)
    children = check_fork(mx, cache, refs, table, lens, [1, 1, 0, 6, 2, 3, 4, 4, 5, -1, 7, 1])
    again = check_fork(mx, cache, refs, children, [2 * page + 5] * 12, [0, 1, 0])
    for t, n in ((table, 7), (children, 12), (again, 3)):
        check_resize(mx, cache, refs, t, [0] * n)
    assert refs == [0] * pages


def test_fork_of_many(mx):
    """More children than a step of the workgroup, more pages than a scan."""
    cache = cache_of(mx, 0, 12000, 1, 16, 32)
    lens = [16 * 40 + 3, 16 * 70, 9]
    refs, table = [0] * 12000, [[-1] * 70 for _ in lens]
    resize(refs, table, lens, 16)
    rng = random.Random(2)
    out = torch.full((5000, 80), 5, dtype=I32, device="cuda")[:, 3:73]
    check_fork(mx, cache, refs, table, lens, [rng.choice([0, 0, 1, 2]) for _ in range(5000)], out=out)


def test_fork_without_enough(mx):
    cache = cache_of(mx, 1, 9, 2, 16, 64)
    lens = [20, 40, 5]
    refs, table = [0] * 9, [[-1] * 2 for _ in lens]  # a row that is too short for its length
    table[0], table[1], table[2] = [4, 2], [0, -1], [1 << 20, 3]
    for p in (4, 2, 0, 3):
        refs[p] = 1
    check_fork(mx, cache, refs, table, lens, [0, 1, 2, 0, 0, 0, 0])
    empty, missing = mx.mx_cache_fork(cache, i32(refs), i32(table), i32(lens), i32([]))
    assert tuple(empty.shape) == (0, 2) and missing.tolist() == []
    rows, missing = mx.mx_cache_fork(cache, i32(refs), i32([]).reshape(0, 2), i32([]), i32([0, -1]))
    assert rows.tolist() == [[-1, -1]] * 2 and missing.tolist() == [0, 0]


# ---- compaction -------------------------------------------------------------------------


def check_compact(mx, cache, starts, keep, counts, table):
    data = snapshot(cache)
    width = max((len(k) for k in keep), default=0)
    k = torch.full((len(keep), width + 3), 1 << 20, dtype=I32)
    for b, row in enumerate(keep):
        k[b, 1:1 + len(row)] = torch.tensor(row, dtype=I32)
    k = k.cuda()[:, 1:1 + width]
    got = mx.mx_cache_compact(cache, i32(starts), k, i32(counts), grid(table))
    want = compact(data, starts, [row + [1 << 20] * (width - len(row)) for row in keep], counts, table, cache.page,
                   cache.pages)
    assert got.dtype == I32 and got.tolist() == want
    same(cache, data)


def tables(rng, sequences, cols, pages):
    order = list(range(pages))
    rng.shuffle(order)
    return [order[b * cols:(b + 1) * cols] for b in range(sequences)]


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("heads,page,dim", [(1, 16, 32), (3, 16, 96), (2, 64, 128), (1, 32, 160), (2, 16, 256), (1, 16, 224)])
def test_compact_paths(mx, fmt, heads, page, dim):
    """Paths of trees at the ends of sequences, as verification gives them."""
    rng = random.Random(dim + page)
    cols = 128 // page + 1
    cache = cache_of(mx, fmt, 6 * cols + 1, heads, page, dim)
    keep, starts, counts = [], [], []
    for b, n in enumerate([1, 2, 13, 40, 64, 70]):
        path = [0] + sorted(rng.sample(range(1, n), min(n - 1, n // 2)))
        keep.append(path + [-1] * (n - len(path)))
        counts.append([len(path), 0, len(path), len(path), 200, 3][b])
        starts.append(rng.randint(0, cols * page - n))
    check_compact(mx, cache, starts, keep, counts, tables(rng, 6, cols, 6 * cols + 1))


@pytest.mark.parametrize("fmt,dim", [(0, 64), (1, 128), (1, 32)])
def test_compact_long(mx, fmt, dim):
    """Whole contexts, more than a group of the workgroup, kept in part, all of them, or shifted by one."""
    rng = random.Random(dim)
    page, cols = 64, 90
    cache = cache_of(mx, fmt, 4 * cols, 2, page, dim)
    n = page * cols
    keep = [sorted(rng.sample(range(n), n // 3)), list(range(n)), list(range(1, n)),
            [i + (i > 2500) + 3 * (i > 5000) for i in range(n - 4)]]
    check_compact(mx, cache, [0, 0, 0, 0], keep, [len(k) for k in keep], tables(rng, 4, cols, 4 * cols))


def test_compact_any_order(mx):
    """Lists in no order, with an entry twice: place i gets what place keep[i] >= i held; others are skipped, and so are
    places without a page."""
    rng = random.Random(7)
    page, cols, n = 16, 400, 5000
    cache = cache_of(mx, 1, 3 * cols, 1, page, 64)
    table = tables(rng, 3, cols, 3 * cols)
    table[1][5], table[1][100], table[2][0] = -1, 3 * cols, 1 << 30
    keep = [[rng.randint(i, n + 200) for i in range(n)] for _ in range(3)]
    for k in keep:
        for i in rng.sample(range(n), 200):
            k[i] = rng.choice([-1, i - 1, -(1 << 31), (1 << 31) - 1, n - 1])
    check_compact(mx, cache, [600, 1300, 3], keep, [n, n - 7, n + 50], table)
    check_compact(mx, cache, [-40, page * cols, 100], keep, [300, 40, -5], table)


def test_compact_nothing(mx):
    cache = cache_of(mx, 1, 4, 1, 16, 64)
    check_compact(mx, cache, [3, 9], [[], []], [5, 0], [[0, 1], [2, 3]])
    check_compact(mx, cache, [], [], [], [])
    none = mx.mx_cache_compact(cache, i32([7]), i32([[1, 2]]), i32([2]), i32([]).reshape(1, 0))
    assert none.tolist() == [9]


# ---- far pages and two calls at once -----------------------------------------------------------


def test_pages_behind_4_gib(mx):
    """Every call on pages whose bytes lie beyond 2^32 of each tensor."""
    page, heads, dim, pages = 64, 8, 128, 70000  # 64 KiB a page
    cache = mx.MXCache.allocate(1, pages, heads, page, dim)
    refs = torch.ones(pages, dtype=I32, device="cuda")
    refs[66000:66003] = 0
    refs[69990:69994] = 0
    table = torch.full((2, 4), -1, dtype=I32, device="cuda")
    missing = mx.mx_cache_resize(cache, refs, table, i32([200, 0]))
    assert table.tolist() == [[66000, 66001, 66002, 69990], [-1] * 4] and not bool(missing.any())
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = [66000, 66001, 66002, 69990]
    for n in NAMES:
        t = getattr(cache, n)
        for p in rows:
            t[p] = torch.randint(0, 256, t[p].shape, generator=g, device="cuda", dtype=torch.uint8)
    old = {n: getattr(cache, n)[rows].clone() for n in NAMES}
    child, missing = mx.mx_cache_fork(cache, refs, table, i32([200, 0]), i32([0]))
    assert child.tolist() == [[66000, 66001, 66002, 69991]] and missing.tolist() == [0]
    mx.mx_cache_copy(cache, i32([66001, 69990]), i32([69992, 69993]))
    keep = i32([[0, 70, 191, 199]])
    assert mx.mx_cache_compact(cache, i32([0]), keep, i32([4]), table[:1]).tolist() == [4]
    for n in NAMES:
        t = getattr(cache, n)
        assert torch.equal(t[[69992, 69993]], old[n][[1, 3]])
        for r in range(64):
            last = token(t, n, 69991, r)
            assert torch.equal(last, token(old[n], n, 3, r)) if r < 8 else not bool(last.any())
        for i, k in enumerate([0, 70, 191, 199]):
            assert torch.equal(token(t, n, 66000, i), token(old[n], n, k // 64, k % 64))
        assert torch.equal(token(t, n, 66000, 4), token(old[n], n, 0, 4)) and torch.equal(t[69990], old[n][3])


def test_two_caches_on_two_streams(mx):
    """Calls on caches and counts of their own may be under way together."""
    both = []
    for k in range(2):
        cache = cache_of(mx, k, 300, 2, 16, 64, seed=k)
        refs, table, lens = [0] * 300, [[-1] * 9 for _ in range(5)], [100, 33, 64, 7, 144]
        resize(refs, table, lens, 16)
        args = i32(refs), grid(table), i32(lens), i32([4, 4, 0, 1, 2, 2])
        both.append((cache, refs, table, lens, snapshot(cache), args, i32([0] * 6), torch.cuda.Stream()))
    torch.cuda.synchronize()
    last = [None, None]
    for turn in range(4):
        for k, (cache, _, _, _, _, args, none, stream) in enumerate(both):
            with torch.cuda.stream(stream):
                last[k], _ = mx.mx_cache_fork(cache, *args)
                if turn < 3:
                    mx.mx_cache_resize(cache, args[0], last[k], none)
    torch.cuda.synchronize()
    for k, (cache, refs, table, lens, data, args, _, _) in enumerate(both):
        want, _ = fork(refs, table, lens, args[3].tolist(), 16, data)
        assert last[k].tolist() == want and args[0].tolist() == refs
        same(cache, data)


# ---- graphs ---------------------------------------------------------------------------------


def test_streams_and_replays(mx):
    """A step of a search, captured: the branches of the step before are freed, new ones forked, a page copied, tokens
    compacted.  Every replay gives what the plain forms give."""
    page, pages = 16, 200
    cache = cache_of(mx, 1, pages, 2, page, 64)
    lens = [100, 37, 16]
    refs, table = [0] * pages, [[-1] * 8 for _ in lens]
    resize(refs, table, lens, page)
    r, t, n = i32(refs), i32(table), i32(lens)
    parents = i32([0, 0, 1, 2, 1])
    branches = torch.full((5, 8), -1, dtype=I32, device="cuda")
    none, keep = torch.zeros(5, dtype=I32, device="cuda"), i32([[0, 2, 3, 3 + 9]] * 3)
    starts, counts, src, dst = i32([80, 20, 0]), i32([4, 2, 3]), i32([150, 151]), i32([160, 161])

    def step():
        mx.mx_cache_resize(cache, r, branches, none)
        _, missing = mx.mx_cache_fork(cache, r, t, n, parents, out=branches)
        mx.mx_cache_copy(cache, src, dst)
        return missing, mx.mx_cache_compact(cache, starts, keep, counts, t)

    def plain(data, held):
        resize(refs, held, [0] * 5, page)
        held, lack = fork(refs, table, lens, parents.tolist(), page, data)
        for a, b in ((150, 160), (151, 161)):
            for name in NAMES:
                data[name][b] = data[name][a]
        return held, lack, compact(data, starts.tolist(), keep.tolist(), counts.tolist(), table, page, pages)

    data, held = snapshot(cache), branches.tolist()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    held, _, _ = plain(data, held)
    same(cache, data)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        missing, after = step()
    for k in range(3):
        parents.copy_(torch.tensor([[0, 0, 1, 2, 1], [2, 2, 2, 1, 0], [-1, 1, 1, 1, 0]][k]))
        graph.replay()
        torch.cuda.synchronize()
        held, lack, lens_after = plain(data, held)
        assert branches.tolist() == held and missing.tolist() == lack and after.tolist() == lens_after
        assert r.tolist() == refs
        same(cache, data)
