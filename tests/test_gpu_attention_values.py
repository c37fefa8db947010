"""Values that are not finite, in attention over the paged MX cache: a row that sees one gets it, whatever else is
special about the token's tile, and no other row does."""
import pytest
import torch

from _attentionref import check
from test_gpu_cache_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from microscaling_quantize_dequantize_amd import binding
    return binding


# rows of a key/value head: few, as many as the few-rows kernel takes at most, many
ROWS = [(4, 1), (2, 3), (8, 4), (8, 12), (5, 60)]


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dim,page", [(64, 16), (96, 32), (128, 16), (256, 32)])
@pytest.mark.parametrize("group,nq", ROWS)
def test_nan_beside_a_page_outside_the_cache(mx, fmt, dim, page, group, nq):
    """A prefix's tile of 64 tokens has a page that is not in the cache, and beside it one with NaN values."""
    c = Case(mx, fmt, 2, group, dim, page, [700, 90 + nq], [nq, nq], seed=dim + nq)
    for b, tok in ((0, 5), (0, 300), (1, 3)):
        p = int(c.table[b, tok // page])
        c.table[b, tok // page + 1] = -1  # the page after it, of the same tile
        c.cache.v_scales[p, 1, dim // 32 - 1, tok % page] = 255
        if fmt == 1:
            c.cache.v_codes[p, 0, tok % page, 7] = 0x7F
    out = c.run(mx)
    check(c, out)
    assert bool(torch.isnan(out).any()) and not bool(torch.isnan(out).all())


def infinite(c, b, tok, head, group, positive):
    """A value of token tok beyond fp32's range in the first dimension of a group of 32, the others of it zero."""
    page = c.cache.page
    p, r = int(c.table[b, tok // page]), tok % page
    fmt, dim = c.cache.fmt, c.cache.dim
    cols = dim // 2 if fmt == 0 else dim
    each = cols * 32 // dim
    codes = torch.zeros(each, dtype=torch.uint8, device="cuda")
    codes[0] = (0x7 if positive else 0xF) if fmt == 0 else (0x7E if positive else 0xFE)
    c.cache.v_codes[p, head, r, group * each:(group + 1) * each] = codes
    c.cache.v_scales[p, head, group, r] = 254


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("group,nq", ROWS)
@pytest.mark.parametrize("tree", [False, True])
def test_infinite_values(mx, fmt, dim, group, nq, tree):
    """A code times its scale beyond the range is an infinity of its sign in every row that sees it, before the new
    tokens or among them, and NaN where both signs meet."""
    c = Case(mx, fmt, 3, group, dim, 16, [1100, 70 + nq], [nq, nq], seed=dim + nq)
    if tree:
        c.random_tree()
    for b, kv in enumerate(c.kv):
        infinite(c, b, 20, 0, 0, True)             # before the new tokens
        infinite(c, b, kv - nq, 1, 1, False)       # the first new token
        infinite(c, b, kv - 1 - nq // 2, 1, 0, True)
        infinite(c, b, 40, 2, 1, True)             # both signs
        infinite(c, b, kv - 1, 2, 1, False)
    out = c.run(mx)
    check(c, out)
    assert bool(torch.isinf(out).any())
