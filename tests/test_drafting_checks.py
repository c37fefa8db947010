"""Refusals of the calls with several axes, of attention to another sequence, of the cache's pages and of verification:
the C entry points on the host (fake addresses, nothing is launched) and the binding's checks."""
import ctypes

import pytest
import torch

from test_cache_checks import (A, EALIGN, EARG, EDTYPE, ELAYOUT, ENULL, ESHAPE, EFMT, OK, NoCompute,  # noqa: F401
                               b, bf, ints, mx, struct)

I32 = torch.int32


def rope(b, **kw):
    f = dict(src=A, st=128, sh=64, dtype=0, tokens=4, heads=2, dim=64, pos=A, stride=4, count=3, axes=A, inv=A, rot=64,
             layout=0, scale=1.0, inverse=0, dst=2 * A, dt=128, dh=64)
    return b.raw().mx_rope_axes(*{**f, **kw}.values())


def test_rope_axes_refusals(b):
    assert rope(b, count=0) == EARG
    assert rope(b, count=1 << 31) == EARG
    assert rope(b, axes=None) == ENULL
    assert rope(b, axes=A + 2) == EALIGN
    assert rope(b, axes=None, rot=0, dst=A) == OK  # in place, nothing to rotate
    assert rope(b, dtype=2) == EDTYPE
    assert rope(b, tokens=-1) == ESHAPE
    assert rope(b, dim=4097) == ESHAPE
    assert rope(b, rot=66) == EARG
    assert rope(b, layout=2) == ELAYOUT
    for name in ("src", "dst", "pos", "inv"):
        assert rope(b, **{name: None}) == ENULL
    assert rope(b, pos=A + 4) == EALIGN
    assert rope(b, dst=A, dt=192) == EARG
    assert rope(b, tokens=0, src=None, dst=None) == OK


def test_write_axes_refusals(b):
    keep = struct(b)

    def write(**kw):
        f = dict(c=ctypes.addressof(keep), k=A, kt=128, kh=64, v=A, vt=128, vh=64, slots=A, tokens=4, pos=A, stride=4,
                 count=2, axes=A, inv=A, rot=64, layout=0, scale=1.0)
        return b.raw().mx_cache_write_axes(*{**f, **kw}.values())

    assert write(c=None) == ENULL
    assert write(count=0) == EARG
    assert write(axes=None) == ENULL
    assert write(axes=A + 1) == EALIGN
    assert write(rot=66) == EARG
    assert write(tokens=-1) == ESHAPE
    for name in ("k", "v", "slots", "pos", "inv"):
        assert write(**{name: None}) == ENULL
    assert write(tokens=0, k=None, v=None, slots=None) == OK


def test_cross_attention_refusals(b):
    keep = struct(b)

    def attend(**kw):
        f = dict(c=ctypes.addressof(keep), q=A, qt=256, qh=64, heads=4, starts=A, lens=A, batch=2, table=A, stride=4,
                 pages=4, total=2, max_q=1, max_kv=64, scale=0.125, out=A, space=A, size=1 << 30)
        return b.raw().mx_cache_cross_attention(*{**f, **kw}.values())

    assert attend(c=None) == ENULL
    assert attend(heads=3) == ESHAPE
    assert attend(max_kv=(1 << 31) - 1) == ESHAPE
    assert attend(stride=3) == ESHAPE
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert attend(scale=scale) == EARG
    for name in ("q", "starts", "lens", "table", "out"):
        assert attend(**{name: None}) == ENULL
    assert attend(q=A + 8) == EALIGN
    space = b.raw().mx_cache_cross_attention_workspace
    need = space(ctypes.addressof(keep), 4, 2, 2, 1, 100000)
    assert need > 0
    assert attend(max_kv=100000, pages=8000, stride=8000, size=need - 1) == EARG
    assert attend(max_kv=100000, pages=8000, stride=8000, space=None) == ENULL
    assert attend(max_kv=100000, pages=8000, stride=8000, space=A + 8) == EALIGN
    assert space(ctypes.addressof(keep), 4, 0, 0, 0, 1000) == 0
    assert space(ctypes.addressof(struct(b, dim=32)), 4, 2, 2, 1, 64) == EARG
    assert attend(total=0, q=None, out=None) == OK


def test_page_refusals(b):
    keep = struct(b)
    c, lib = ctypes.addressof(keep), b.raw()
    nothing = struct(b, pages=0, k_codes=None, k_scales=None, v_codes=None, v_scales=None)
    n = ctypes.addressof(nothing)

    def copy(**kw):
        return lib.mx_cache_copy(*{**dict(c=c, src=A, dst=A, count=3), **kw}.values())

    def resize(**kw):
        f = dict(c=c, refs=A, table=A, stride=4, pages=4, lens=A, rows=2, missing=A)
        return lib.mx_cache_resize(*{**f, **kw}.values())

    def fork(**kw):
        f = dict(c=c, refs=A, table=A, stride=4, pages=4, lens=A, rows=2, parents=A, children=3, out=A, out_stride=4,
                 missing=A)
        return lib.mx_cache_fork(*{**f, **kw}.values())

    def compact(**kw):
        f = dict(c=c, starts=A, keep=A, keep_stride=5, most=5, counts=A, table=A, stride=4, pages=4, batch=2, lens=A)
        return lib.mx_cache_compact(*{**f, **kw}.values())

    bad = struct(b, fmt=3)
    for call in (copy, resize, fork, compact):
        assert call(c=None) == ENULL
        assert call(c=ctypes.addressof(bad)) == EFMT
    assert copy(count=-1) == ESHAPE
    assert copy(count=1 << 24) == ESHAPE
    assert copy(src=None) == ENULL and copy(dst=None) == ENULL
    assert copy(src=A + 2) == EALIGN and copy(dst=A + 1) == EALIGN
    assert copy(count=0, src=None, dst=None) == OK
    assert copy(c=n) == OK
    for call in (resize, fork):
        assert call(rows=-1) == ESHAPE
        assert call(rows=(1 << 24) + 1) == ESHAPE
        assert call(stride=3) == ESHAPE
        assert call(pages=-1) == ESHAPE
        assert call(pages=1 << 28, stride=1 << 28, **({"out_stride": 1 << 28} if call is fork else {})) == ESHAPE
        for name in ("refs", "table", "lens", "missing"):
            assert call(**{name: None}) == ENULL
            assert call(**{name: A + 2}) == EALIGN
    assert resize(rows=0, refs=None, table=None, lens=None, missing=None) == OK
    assert fork(children=-1) == ESHAPE
    assert fork(children=1 << 22) == ESHAPE  # with two heads
    assert fork(out_stride=3) == ESHAPE
    assert fork(parents=None) == ENULL and fork(out=None) == ENULL
    assert fork(parents=A + 1) == EALIGN and fork(out=A + 2) == EALIGN
    assert fork(children=0, parents=None, out=None, missing=None) == OK
    assert compact(batch=-1) == ESHAPE
    assert compact(batch=1 << 19) == ESHAPE
    assert compact(keep_stride=4) == ESHAPE
    assert compact(most=-1) == ESHAPE
    assert compact(stride=3) == ESHAPE
    for name in ("starts", "keep", "counts", "table", "lens"):
        assert compact(**{name: None}) == ENULL
        assert compact(**{name: A + 2}) == EALIGN
    assert compact(batch=0, starts=None, keep=None, counts=None, table=None, lens=None) == OK


def test_verify_refusals(b):
    lib = b.raw()

    def verify(**kw):
        f = dict(target=A, ts=100, draft=A, ds=100, dtype=0, vocab=100, tokens=A, uniforms=A, starts=A, parents=A, batch=2,
                 total=9, max_q=5, counts=A, path=A, out=A, space=A, size=1 << 40)
        return lib.mx_verify(*{**f, **kw}.values())

    assert verify(dtype=2) == EDTYPE
    assert verify(vocab=0) == ESHAPE
    assert verify(vocab=(1 << 30) + 1) == ESHAPE
    assert verify(batch=-1) == ESHAPE
    assert verify(batch=1 << 22) == ESHAPE
    assert verify(total=-1) == ESHAPE
    assert verify(total=1 << 31) == ESHAPE
    assert verify(max_q=-1) == ESHAPE
    assert verify(max_q=1025) == ESHAPE
    for name in ("target", "tokens", "uniforms", "starts", "counts", "path", "out"):
        assert verify(**{name: None}) == ENULL
    for name, off in (("target", 1), ("draft", 1), ("tokens", 4), ("uniforms", 4), ("starts", 2), ("parents", 2),
                      ("counts", 2), ("path", 2), ("out", 4)):
        assert verify(**{name: A + off}) == EALIGN
    assert verify(dtype=1, target=A + 2) == EALIGN
    assert verify(batch=0, target=None, starts=None, counts=None) == OK
    assert lib.mx_verify_workspace(2, 9, 1025, 100) == ESHAPE
    assert lib.mx_verify_workspace(0, 0, 0, 1) >= 0
    need = lib.mx_verify_workspace(2, 9, 5, 200000)
    if need:
        assert verify(vocab=200000, size=need - 1) == EARG
        assert verify(vocab=200000, space=None) == ENULL
        assert verify(vocab=200000, space=A + 8) == EALIGN


# ---- binding -------------------------------------------------------------------


def test_binding_axes(mx):
    f = torch.zeros(32, dtype=torch.float64)
    x = bf(5, 2, 64)
    for positions, axes in ((ints(5), ints(32, dtype=I32)), (ints(3, 4), ints(32, dtype=I32)), (ints(3, 5), ints(32)),
                            (ints(3, 5), ints(31, dtype=I32)), (ints(3, 5, dtype=I32), ints(32, dtype=I32)),
                            (ints(0, 5), ints(32, dtype=I32)), (ints(5, 3).t(), ints(32, dtype=I32)),
                            (ints(3, 5), ints(32, 1, dtype=I32))):
        with pytest.raises(ValueError):
            mx.mx_rope(x, positions, f, axes=axes)
    cache = mx.MXCache.allocate(1, 2, 2, 16, 64, device="cpu")
    with pytest.raises(ValueError, match="axes need positions"):
        mx.mx_cache_write(cache, x, x, ints(5), axes=ints(32, dtype=I32))
    with pytest.raises(ValueError):
        mx.mx_cache_write(cache, x, x, ints(5), positions=ints(5), inv_freq=f, axes=ints(32, dtype=I32))


def test_binding_cross_attention(mx, monkeypatch):
    real = mx._lib.real
    monkeypatch.setattr(NoCompute, "mx_cache_cross_attention_workspace",
                        property(lambda self: real.mx_cache_cross_attention_workspace), raising=False)
    cache = mx.MXCache.allocate(1, 2, 3, 16, 64, device="cpu")
    good = dict(q=bf(4, 6, 64), q_starts=ints(3, dtype=I32), kv_lens=ints(2, dtype=I32),
                block_table=ints(2, 2, dtype=I32), max_q=2, max_kv=20)
    for kw in (dict(q=bf(4, 5, 64)), dict(q=bf(4, 6, 32)), dict(q_starts=ints(3)), dict(kv_lens=ints(2)),
               dict(block_table=ints(3, 2, dtype=I32)), dict(out=bf(4, 6, 63))):
        with pytest.raises(ValueError):
            mx.mx_cache_cross_attention(cache, **{**good, **kw})
    with pytest.raises(TypeError):
        mx.mx_cache_cross_attention(None, **good)


def test_binding_pages(mx):
    cache = mx.MXCache.allocate(1, 6, 3, 16, 64, device="cpu")
    refs, table, lens = ints(6, dtype=I32), ints(2, 4, dtype=I32), ints(2, dtype=I32)
    for src, dst in ((ints(2), ints(2, dtype=I32)), (ints(2, dtype=I32), ints(3, dtype=I32)),
                     (ints(2, 1, dtype=I32), ints(2, dtype=I32)), (None, ints(2, dtype=I32))):
        with pytest.raises(ValueError):
            mx.mx_cache_copy(cache, src, dst)
    for args in ((refs[:5], table, lens), (refs.long(), table, lens), (refs, table[:1], lens), (refs, table.long(), lens),
                 (refs, table, ints(2)), (refs, ints(4, 2, dtype=I32).t(), lens), (refs, table, None)):
        with pytest.raises(ValueError):
            mx.mx_cache_resize(cache, *args)
    parents = ints(3, dtype=I32)
    for args, out in (((refs, table, lens, parents.long()), None), ((refs, table, ints(3, dtype=I32), parents), None),
                      ((refs, table, lens, parents), ints(3, 5, dtype=I32)),
                      ((refs, table, lens, parents), ints(2, 4, dtype=I32)),
                      ((refs, table, lens, parents), ints(3, 4))):
        with pytest.raises(ValueError):
            mx.mx_cache_fork(cache, *args, out=out)
    whole = ints(5, 4, dtype=I32)
    with pytest.raises(ValueError, match="overlap"):
        mx.mx_cache_fork(cache, refs, whole[:2], lens, parents, out=whole[1:4])
    keep = ints(2, 3, dtype=I32)
    for args in ((lens, keep, lens, table[:1]), (lens, keep[:1], lens, table), (lens, keep.long(), lens, table),
                 (lens.long(), keep, lens, table), (lens, keep, ints(3, dtype=I32), table), (keep, keep, lens, table)):
        with pytest.raises(ValueError):
            mx.mx_cache_compact(cache, *args)
    with pytest.raises(TypeError):
        mx.mx_cache_copy(None, lens, lens)


def test_binding_verify(mx, monkeypatch):
    real = mx._lib.real
    monkeypatch.setattr(NoCompute, "mx_verify_workspace", property(lambda self: real.mx_verify_workspace), raising=False)
    p = torch.zeros(7, 50)
    good = dict(target=p, tokens=ints(7), uniforms=torch.zeros(7, dtype=torch.float64), q_starts=ints(3, dtype=I32),
                max_q=5)
    for kw in (dict(target=p.half()), dict(target=p[0]), dict(target=torch.zeros(50, 7).t()), dict(tokens=ints(6)),
               dict(tokens=ints(7, dtype=I32)), dict(uniforms=torch.zeros(7)), dict(q_starts=ints(3)),
               dict(q_starts=ints(0, dtype=I32)), dict(draft=torch.zeros(7, 49)), dict(draft=p.bfloat16()),
               dict(draft=torch.zeros(50, 7).t()), dict(parents=ints(7)), dict(parents=ints(6, dtype=I32))):
        with pytest.raises(ValueError):
            mx.mx_verify(**{**good, **kw})
    with pytest.raises(TypeError):
        mx.mx_verify(**{**good, "target": None})
    for kw in (dict(max_q=1025), dict(max_q=-1), dict(target=torch.zeros(7, 0))):
        with pytest.raises(mx.MXError):
            mx.mx_verify(**{**good, **kw})
