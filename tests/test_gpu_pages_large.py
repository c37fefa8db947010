"""The cache's pages at sizes where the calls take other paths: copies around 64 MiB, compaction of contexts whose tables
are longer than what a workgroup holds of them and of tokens whose pieces are no power of two, forks of many heads over
several steps."""
import random

import pytest
import torch

from test_gpu_pages import I32, NAMES, cache_of, check_fork, check_resize, i32, mx, resize, same, snapshot  # noqa: F401

pytestmark = pytest.mark.gpu


# (bytes of keys and values of a page: 135168, 9792 and 29568; from 2^26 bytes on a copy is written past the caches)
@pytest.mark.parametrize("fmt,heads,page,dim,each", [(1, 8, 64, 128, 135168), (0, 3, 32, 96, 9792), (1, 7, 16, 128, 29568)])
@pytest.mark.parametrize("above", [False, True])
def test_copies_around_64_mib(mx, fmt, heads, page, dim, each, above):
    count = -(-(1 << 26) // each) - (not above)
    pages = 2 * count + 3
    cache = cache_of(mx, fmt, pages, heads, page, dim, seed=count)
    assert each == sum(getattr(cache, n)[0].numel() for n in NAMES)
    want = snapshot(cache)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(count))
    src, dst = order[:count], order[count:2 * count]
    for n in NAMES:
        want[n][dst] = want[n][src]
    src, dst = src.to(I32), dst.to(I32)
    src[5], dst[7] = -1, pages  # two pairs that are skipped
    for n in NAMES:
        old = getattr(cache, n).cpu()
        want[n][order[count + 5]], want[n][order[count + 7]] = old[order[count + 5]], old[order[count + 7]]
    mx.mx_cache_copy(cache, src.cuda(), dst.cuda())
    same(cache, want)


def moved(data, start, keep, table, page):
    """What compaction makes of one sequence: places start + i get what places start + keep[i] hold (every place has a
    page)."""
    def at(place):
        return table[place // page], place % page

    i = torch.arange(len(keep))
    use = keep >= i
    (sp, sr), (dp, dr) = at(start + keep[use]), at(start + i[use])
    for n in NAMES:
        t = data[n]
        if n.endswith("codes"):
            t[dp, :, dr] = t[sp, :, sr].clone()
        else:
            t[dp, :, :, dr] = t[sp, :, :, sr].clone()


def check_moved(mx, cache, starts, keep, table):
    data = snapshot(cache)
    most = max(len(k) for k in keep)
    lists = torch.full((len(keep), most), 1 << 20, dtype=I32)
    for b, k in enumerate(keep):
        lists[b, :len(k)] = k.to(I32)
    counts = [len(k) for k in keep]
    got = mx.mx_cache_compact(cache, i32(starts), lists.cuda(), i32(counts), table.to(I32).cuda())
    for b, k in enumerate(keep):
        moved(data, starts[b], k, table[b], cache.page)
    assert got.tolist() == [s + n for s, n in zip(starts, counts)]
    same(cache, data)


def some_of(n, kept, seed):
    return torch.randperm(n, generator=torch.Generator().manual_seed(seed))[:kept].sort()[0]


@pytest.mark.parametrize("fmt,dim", [(0, 96), (1, 64)])
@pytest.mark.parametrize("start", [0, 16 * 130 + 5])
def test_compact_behind_the_table_that_is_held(mx, fmt, dim, start):
    """4500 pages of 16 tokens: sources and places lie on both sides of entry 4096 from the first one on."""
    cols, page = 4500, 16
    cache = cache_of(mx, fmt, cols + 7, 1, page, dim, seed=start)
    table = torch.randperm(cols + 7, generator=torch.Generator().manual_seed(dim))[None, :cols]
    n = cols * page - start
    dense = some_of(n, n - 1500, 1)
    assert int(dense[-1]) > 4096 * page + 1000 and len(dense) > 4096 * page + 1000
    check_moved(mx, cache, [start], [dense], table)
    few = torch.tensor([0, 3, 4096 * page - 1, 4096 * page, 4097 * page + 1, n - 1])  # in the small workgroups
    check_moved(mx, cache, [start], [few], table)


@pytest.mark.parametrize("fmt,dim", [(0, 96), (1, 96), (0, 160), (1, 160), (0, 224), (1, 224), (0, 32), (1, 256)])
@pytest.mark.parametrize("batch,heads", [(1, 1), (3, 2), (40, 4)])
def test_compact_pieces(mx, fmt, dim, batch, heads):
    """Long lists; a token has 1 to 16 pieces, which few heads share among workgroups and many do not."""
    page, cols = 32, 200 if batch < 40 else 160
    n = page * cols - 9
    cache = cache_of(mx, fmt, batch * cols, heads, page, dim, seed=dim)
    table = torch.randperm(batch * cols, generator=torch.Generator().manual_seed(dim)).reshape(batch, cols)
    keep = [some_of(n, n - n // (b % 3 + 2), b) for b in range(batch)]
    check_moved(mx, cache, [b % 9 for b in range(batch)], keep, table)


def test_fork_of_many_heads(mx):
    """2600 children, 5 heads: more rows than a step of the workgroup that hands pages out, and a copy for each head."""
    page, cols = 32, 6
    cache = cache_of(mx, 1, 6000, 5, page, 32, seed=9)
    lens = [32 * 5 + 7, 32 * 2, 31, 0, 32 * 3 + 1]
    refs, table = [0] * 6000, [[-1] * cols for _ in lens]
    resize(refs, table, lens, page)
    rng = random.Random(4)
    children = check_fork(mx, cache, refs, table, lens, [rng.choice([0, 1, 2, 3, 4, 4, -1, 5]) for _ in range(2600)])
    check_resize(mx, cache, refs, children, [0] * 2600)
    check_resize(mx, cache, refs, table, [0] * 5)
    assert refs == [0] * 6000
