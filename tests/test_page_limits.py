"""Tables of pages whose missing entries 32 bits do not count: refused on the host (fake addresses, nothing is
launched)."""
import ctypes

from test_cache_checks import A, ESHAPE, ENULL, b, mx, struct  # noqa: F401


def test_tables_of_too_many_entries(b):
    keep = struct(b, page=16)

    def resize(rows, pages, **kw):
        f = dict(c=ctypes.addressof(keep), refs=A, table=A, stride=pages, pages=pages, lens=A, rows=rows, missing=A)
        return b.raw().mx_cache_resize(*{**f, **kw}.values())

    # 1024 rows of 2^21 entries are 2^31 (what lies within the limits goes on to the next check, of a null pointer)
    assert resize(1024, 1 << 21) == ESHAPE
    assert resize(1 << 24, 1 << 21) == ESHAPE
    assert resize(17, (1 << 27) - 1) == ESHAPE
    assert resize(1024, (1 << 21) - 1, refs=None) == ENULL
    assert resize(1 << 24, (1 << 21) - 1, refs=None) == ENULL
    assert resize(16, (1 << 27) - 1, refs=None) == ENULL
