"""Refusals of the rotary, cache and attention calls: the C entry points on the
host (fake addresses, nothing is launched) and the binding's checks of shapes,
types and strides (host tensors; the library's calls are replaced by a stub)."""
import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "microscaling_quantize_dequantize_amd", "libmxqdq.so")
OK, EFMT, EDTYPE, ESHAPE, ENULL, EALIGN, ELAYOUT, EARG = 0, -1, -2, -3, -5, -6, -8, -9
A = 1 << 20  # a 16-byte aligned fake address; never dereferenced


@pytest.fixture(scope="module")
def b():
    if not os.path.exists(LIB):
        from microscaling_quantize_dequantize_amd import build
        build.build()
    from microscaling_quantize_dequantize_amd import binding
    return binding


def struct(b, **kw):
    f = dict(fmt=1, heads=2, page=16, dim=64, pages=4, k_codes=A, k_scales=A, v_codes=A, v_scales=A)
    f.update(kw)
    return b._CacheStruct(**f)


def rope(b, **kw):
    f = dict(src=A, st=128, sh=64, dtype=0, tokens=4, heads=2, dim=64, pos=A, inv=A, rot=64, layout=0, scale=1.0,
             inverse=0, dst=2 * A, dt=128, dh=64)
    f.update(kw)
    return b.raw().mx_rope(*f.values())


def test_rope_refusals(b):
    assert rope(b, dtype=2) == EDTYPE
    assert rope(b, tokens=-1) == ESHAPE
    assert rope(b, heads=-1) == ESHAPE
    assert rope(b, dim=4097) == ESHAPE
    assert rope(b, rot=66) == EARG
    assert rope(b, rot=31) == EARG
    assert rope(b, rot=-2) == EARG
    assert rope(b, layout=2) == ELAYOUT
    assert rope(b, src=None) == ENULL
    assert rope(b, dst=None) == ENULL
    assert rope(b, pos=None) == ENULL
    assert rope(b, inv=None) == ENULL
    assert rope(b, src=A + 1) == EALIGN
    assert rope(b, dtype=1, dst=A + 2) == EALIGN
    assert rope(b, inv=A + 4) == EALIGN
    assert rope(b, dst=A, dt=192) == EARG
    assert rope(b, tokens=0, src=None, dst=None) == OK
    assert rope(b, dst=A, rot=0) == OK  # in place, nothing to rotate


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=2), EFMT), (dict(dim=48), ESHAPE), (dict(dim=288), ESHAPE), (dict(dim=0), ESHAPE), (dict(page=8), ESHAPE),
    (dict(page=48), ESHAPE), (dict(page=1 << 17), ESHAPE), (dict(heads=0), ESHAPE), (dict(pages=-1), ESHAPE),
    (dict(pages=1 << 31), ESHAPE), (dict(heads=60000, page=65536, pages=1 << 20), ESHAPE), (dict(k_codes=A + 8), EALIGN),
    (dict(v_scales=A + 4), EALIGN)])
def test_cache_refusals(b, kw, status):
    c = ctypes.addressof(keep := struct(b, **kw))
    lib = b.raw()
    assert lib.mx_cache_write(c, A, 128, 64, A, 128, 64, A, 4, A, A, 64, 0, 1.0) == status
    assert lib.mx_cache_read(c, A, 4, A, A) == status
    assert lib.mx_cache_attention_workspace(c, 4, 1, 1, 1, 16) == status
    del keep


def test_write_and_read_refusals(b):
    lib = b.raw()
    keep = struct(b)
    c = ctypes.addressof(keep)

    def write(**kw):
        f = dict(c=c, k=A, kt=128, kh=64, v=A, vt=128, vh=64, slots=A, tokens=4, pos=A, inv=A, rot=64, layout=0,
                 scale=1.0)
        f.update(kw)
        return lib.mx_cache_write(*f.values())

    assert write(c=None) == ENULL
    assert write(tokens=-1) == ESHAPE
    assert write(rot=66) == EARG
    assert write(rot=3) == EARG
    assert write(layout=-1) == ELAYOUT
    for name in ("k", "v", "slots", "pos", "inv"):
        assert write(**{name: None}) == ENULL
    assert write(k=A + 1) == EALIGN
    assert write(slots=A + 4) == EALIGN
    assert write(tokens=0, k=None, v=None, slots=None) == OK
    assert lib.mx_cache_read(c, A, 4, A + 8, A) == EALIGN
    assert lib.mx_cache_read(c, None, 4, A, A) == ENULL
    assert lib.mx_cache_read(c, A, 4, A, None) == ENULL
    assert lib.mx_cache_read(c, None, 0, None, None) == OK
    empty = struct(b, pages=0, k_codes=None, k_scales=None, v_codes=None, v_scales=None)
    assert lib.mx_cache_write(ctypes.addressof(empty), A, 128, 64, A, 128, 64, A, 4, None, None, 0, 0, 1.0) == OK


def test_attention_refusals(b):
    lib = b.raw()
    keep = struct(b)
    c = ctypes.addressof(keep)

    def attend(**kw):
        f = dict(c=c, q=A, qt=256, qh=64, heads=4, starts=A, lens=A, batch=2, table=A, stride=4, pages=4, total=2,
                 max_q=1, max_kv=64, tree=None, words=0, scale=0.125, out=A, space=A, size=1 << 30)
        f.update(kw)
        return lib.mx_cache_attention(*f.values())

    assert attend(c=None) == ENULL
    assert attend(heads=3) == ESHAPE
    assert attend(heads=0) == ESHAPE
    assert attend(batch=-1) == ESHAPE
    assert attend(total=1 << 31) == ESHAPE
    assert attend(max_q=-1) == ESHAPE
    assert attend(max_kv=(1 << 31) - 1) == ESHAPE
    assert attend(batch=1 << 24, total=1 << 20, max_q=1 << 20) == ESHAPE  # more rows than a grid has workgroups for
    assert attend(stride=3) == ESHAPE
    assert attend(pages=(1 << 31) // 16) == ESHAPE
    assert attend(words=-1) == ESHAPE
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert attend(scale=scale) == EARG
    for name in ("q", "starts", "lens", "table", "out"):
        assert attend(**{name: None}) == ENULL
    for name, off in (("q", 8), ("out", 8), ("starts", 2), ("lens", 2), ("table", 2)):
        assert attend(**{name: A + off}) == EALIGN
    assert attend(tree=A + 4, words=1) == EALIGN
    assert attend(tree=A, words=0) == EARG
    assert attend(tree=A, words=1, total=100, max_q=65) == EARG
    assert attend(qt=252) == EALIGN
    assert attend(qh=68) == EALIGN
    need = lib.mx_cache_attention_workspace(c, 4, 2, 2, 1, 100000)
    assert need > 0
    assert attend(max_kv=100000, size=need - 1) == EARG
    assert attend(max_kv=100000, space=None) == ENULL
    assert attend(max_kv=100000, space=A + 8) == EALIGN
    assert attend(batch=0, q=None, out=None) == OK
    assert attend(total=0, q=None, out=None) == OK
    small = struct(b, dim=32)
    assert lib.mx_cache_attention_workspace(ctypes.addressof(small), 4, 2, 2, 1, 64) == EARG
    nothing = struct(b, pages=0)
    assert attend(c=ctypes.addressof(nothing)) == ENULL
    assert lib.mx_cache_attention_workspace(c, 4, 0, 0, 0, 1000) == 0


# ---- binding -------------------------------------------------------------------


class NoCompute:
    def __init__(self, real):
        self.real = real

    def __getattr__(self, name):
        if name in ("mx_cache_attention_workspace", "mx_status_string"):
            return getattr(self.real, name)
        raise AssertionError(f"{name} was called")


@pytest.fixture
def mx(b, monkeypatch):
    """The binding with host tensors taken for GPU ones and no call let through."""
    monkeypatch.setattr(b, "_lib", NoCompute(b._lib))
    monkeypatch.setattr(b, "_dev", lambda t, name: t.data_ptr())
    monkeypatch.setattr(b, "_place", lambda t, name: None)
    return b


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def ints(*shape, dtype=torch.int64):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_host_tensors(b):
    with pytest.raises(TypeError):
        b.mx_rope(bf(2, 1, 64), ints(2), torch.zeros(32, dtype=torch.float64))
    with pytest.raises(TypeError):
        b.MXCache.allocate(1, 2, 2, 16, 64, device="cpu")
    with pytest.raises(TypeError):
        b.mx_cache_read(None, ints(2))


def test_binding_rope(mx):
    f = torch.zeros(32, dtype=torch.float64)
    for args in ((bf(2, 64), ints(2), f), (bf(2, 1, 64).half(), ints(2), f), (bf(2, 1, 64), ints(3), f),
                 (bf(2, 1, 64), ints(2, dtype=torch.int32), f), (bf(2, 1, 64), ints(2), f.float()),
                 (bf(2, 64, 2).transpose(1, 2), ints(2), f)):
        with pytest.raises(ValueError):
            mx.mx_rope(*args)
    with pytest.raises(TypeError):
        mx.mx_rope(None, ints(2), f)
    for dst in (bf(2, 1, 63), torch.zeros(2, 1, 64)):
        with pytest.raises(ValueError):
            mx.mx_rope(bf(2, 1, 64), ints(2), f, dst=dst)


def test_binding_cache(mx):
    def u8(*shape):
        return torch.zeros(shape, dtype=torch.uint8)

    good = (u8(2, 3, 16, 64), u8(2, 3, 2, 16), u8(2, 3, 16, 64), u8(2, 3, 2, 16))
    mx.MXCache(1, *good)
    for i, bad in ((0, u8(2, 3, 16, 65)), (0, u8(2, 3, 24, 64)), (0, u8(2, 3, 8, 64)), (1, u8(2, 3, 16, 2)),
                   (2, u8(2, 3, 16, 32)), (3, good[3].int()), (0, u8(2, 3, 64))):
        with pytest.raises(ValueError):
            mx.MXCache(1, *[bad if j == i else t for j, t in enumerate(good)])
    with pytest.raises(ValueError):
        mx.MXCache(2, *good)
    cache = mx.MXCache(1, *good)
    k = bf(5, 3, 64)
    for args in ((bf(5, 2, 64), k, ints(5)), (k, bf(4, 3, 64), ints(5)), (k, k, ints(4)), (k.float(), k, ints(5)),
                 (k, k, ints(5, dtype=torch.int32))):
        with pytest.raises(ValueError):
            mx.mx_cache_write(cache, *args)
    with pytest.raises(ValueError):
        mx.mx_cache_write(cache, k, k, ints(5), positions=ints(5))
    with pytest.raises(ValueError):
        mx.mx_cache_read(cache, ints(5), k=bf(5, 3, 63))
    with pytest.raises(ValueError):
        mx.mx_cache_read(cache, ints(5, 1))


def test_binding_attention(mx):
    cache = mx.MXCache.allocate(1, 2, 3, 16, 64, device="cpu")
    i32 = torch.int32
    good = dict(q=bf(4, 6, 64), q_starts=ints(3, dtype=i32), kv_lens=ints(2, dtype=i32),
                block_table=ints(2, 2, dtype=i32), max_q=2, max_kv=20)
    for kw in (dict(q=bf(4, 5, 64)), dict(q=bf(4, 6, 32)), dict(q=bf(4, 6, 64).float()), dict(q_starts=ints(3)),
               dict(q_starts=ints(2, dtype=i32)), dict(kv_lens=ints(2)), dict(block_table=ints(2, 2)),
               dict(block_table=ints(3, 2, dtype=i32)), dict(block_table=ints(2, 2, dtype=i32).t()[:, :]),
               dict(tree=ints(4)), dict(tree=ints(3, 1)), dict(tree=ints(4, 1), max_q=65),
               dict(tree=ints(4, 1, dtype=i32)), dict(out=bf(4, 6, 63))):
        with pytest.raises(ValueError):
            mx.mx_cache_attention(cache, **{**good, **kw})
    with pytest.raises(mx.MXError):
        mx.mx_cache_attention(cache, **{**good, "max_kv": -1})
