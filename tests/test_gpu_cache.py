"""The paged MX cache on the GPU: codes and scales bit for bit against the
scalar oracle (keys rotated in 64 bits and rounded to bf16 first), read back
exactly; slots out of order, outside the cache, far offsets, strides."""
import pytest
import torch

import _cacheref as R

pytestmark = pytest.mark.gpu
HALF, INTERLEAVED = 0, 1


@pytest.fixture(scope="module")
def mx():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from microscaling_quantize_dequantize_amd import binding
    return binding


def frequencies(pairs):
    return 10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device="cuda") / max(pairs, 1))


def heads_of(g, tokens, heads, dim, pad=0):
    wide = torch.randn((tokens, heads + 1, dim + pad), generator=g, device="cuda")
    wide *= torch.exp2(torch.randint(-8, 8, (tokens, heads + 1, 1), generator=g, device="cuda").float())
    return wide.bfloat16()[:, 1:, :dim]


def filled(mx, fmt, pages, heads, page, dim, seed=0):
    c = mx.MXCache.allocate(fmt, pages, heads, page, dim)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        t.copy_(torch.randint(0, 127, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    return c


def check_write(mx, fmt, tokens, heads, dim, page, rot, layout, pad=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(tokens + 7 * dim + rot)
    pages = -(-tokens // page) + 2
    cache = filled(mx, fmt, pages, heads, page, dim)
    before = {n: getattr(cache, n).clone() for n in ("k_codes", "k_scales", "v_codes", "v_scales")}
    k, v = heads_of(g, tokens, heads, dim, pad), heads_of(g, tokens, heads, dim, pad)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:tokens]
    pos = torch.randint(0, 1 << 20, (tokens,), generator=g, device="cuda")
    f = frequencies(rot // 2)
    if rot:
        mx.mx_cache_write(cache, k, v, slots, positions=pos, inv_freq=f, layout=layout, scale=scale)
        turned = R.rotate(k, pos, f, scale, layout, False)[0].float().bfloat16()
        turned[..., rot:] = k[..., rot:].cpu()
    else:
        mx.mx_cache_write(cache, k, v, slots)
        turned = k.cpu()
    p, r = (slots // page).cpu(), (slots % page).cpu()
    for x, n in ((turned, "k"), (v.cpu(), "v")):
        codes, scales = R.quantise(fmt, x)
        want_c, want_s = before[n + "_codes"].cpu(), before[n + "_scales"].cpu()
        want_c[p, :, r], want_s[p, :, :, r] = codes, scales
        assert torch.equal(getattr(cache, n + "_scales").cpu(), want_s), n
        assert torch.equal(getattr(cache, n + "_codes").cpu(), want_c), n
    rk, rv = mx.mx_cache_read(cache, slots)
    for got, n in ((rk, "k"), (rv, "v")):
        c, s = getattr(cache, n + "_codes").cpu()[p, :, r], getattr(cache, n + "_scales").cpu()[p, :, :, r]
        assert torch.equal(got.cpu(), R.values(fmt, c, s).bfloat16()), n


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("layout", [HALF, INTERLEAVED])
@pytest.mark.parametrize("tokens,heads,dim,page,rot", [
    (1, 1, 32, 16, 32), (1, 8, 128, 64, 128), (17, 5, 96, 16, 32), (33, 3, 64, 32, 0), (130, 2, 256, 128, 254),
    (65, 1, 192, 16, 96), (7, 4, 160, 256, 50), (700, 16, 64, 64, 64)])
def test_write_and_read(mx, fmt, layout, tokens, heads, dim, page, rot):
    check_write(mx, fmt, tokens, heads, dim, page, rot, layout, scale=1.0 if rot % 4 else 1.125)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("layout", [HALF, INTERLEAVED])
@pytest.mark.parametrize("pad", [1, 2, 8])
def test_write_from_strided_rows(mx, fmt, layout, pad):
    check_write(mx, fmt, 21, 3, 64, 16, 48, layout, pad=pad)


@pytest.mark.parametrize("fmt", [0, 1])
def test_slots_outside_the_cache(mx, fmt):
    """They are skipped when written and zeros when read; nothing else changes."""
    cache = filled(mx, fmt, 2, 3, 16, 64, seed=9)
    before = [t.clone() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
    k = torch.randn((5, 3, 64), device="cuda").bfloat16()
    outside = torch.tensor([-1, 32, 1 << 40, -(1 << 40), 33], device="cuda")
    mx.mx_cache_write(cache, k, k, outside)
    for t, b in zip((cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales), before):
        assert torch.equal(t, b)
    rk, rv = mx.mx_cache_read(cache, outside)
    assert not bool(rk.any()) and not bool(rv.any())


@pytest.mark.parametrize("fmt", [0, 1])
def test_special_values(mx, fmt):
    """All-zero and subnormal groups, -0, saturating values; NaN and Inf make their own group NaN and no other."""
    x = torch.zeros((4, 2, 64), device="cuda").bfloat16()
    x[0, 0, 3], x[0, 1, 40] = 1e-39, -0.0
    x[1, 0, :32] = torch.linspace(-3.3e38, 3.3e38, 32).bfloat16().cuda()
    x[2, 1, 5], x[3, 0, 63] = float("nan"), float("-inf")
    cache = mx.MXCache.allocate(fmt, 1, 2, 16, 64)
    slots = torch.tensor([3, 0, 15, 7], device="cuda")
    mx.mx_cache_write(cache, x, x, slots)
    codes, scales = R.quantise(fmt, x.cpu())
    assert torch.equal(cache.v_codes[0][:, slots].transpose(0, 1).cpu(), codes)
    assert torch.equal(cache.v_scales[0][:, :, slots].permute(2, 0, 1).cpu(), scales)
    rk, _ = mx.mx_cache_read(cache, slots)
    # (the difference of linspace's ends passes fp32's range, so group (1, 0, 0) holds NaN as well)
    finite = torch.isfinite(x).unflatten(-1, (2, 32)).all(-1, keepdim=True).expand(4, 2, 2, 32).flatten(-2)
    assert torch.equal(torch.isnan(rk), ~finite), "NaN in another group"
    assert int((~finite).sum()) == 3 * 32


@pytest.mark.parametrize("fmt", [0, 1])
def test_largest_values_saturate(mx, fmt):
    x = torch.zeros((1, 1, 64), device="cuda").bfloat16()
    x[0, 0, :32] = (torch.arange(-16, 16, device="cuda") * (3.3e38 / 16)).bfloat16()
    x[0, 0, 32:] = 1.9921875
    cache = mx.MXCache.allocate(fmt, 1, 1, 16, 64)
    slots = torch.tensor([4], device="cuda")
    mx.mx_cache_write(cache, x, x, slots)
    codes, scales = R.quantise(fmt, x.cpu())
    assert torch.equal(cache.k_codes[0][:, slots].transpose(0, 1).cpu(), codes)
    rk, rv = mx.mx_cache_read(cache, slots)
    assert torch.equal(rk.cpu(), R.values(fmt, codes, scales).bfloat16()) and torch.equal(rk, rv)
    assert bool(torch.isfinite(rk).all())


def test_offsets_past_32_bits(mx):
    """Slots in the last pages of a cache of more than 2^32 bytes of codes."""
    heads, page, dim = 16, 256, 128
    pages = (1 << 32) // (heads * page * dim) + 3
    cache = mx.MXCache.allocate(1, pages, heads, page, dim)
    slots = torch.tensor([pages * page - 1, 5, (pages - 2) * page + 17], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = heads_of(g, 3, heads, dim), heads_of(g, 3, heads, dim)
    mx.mx_cache_write(cache, k, v, slots)
    rk, rv = mx.mx_cache_read(cache, slots)
    for x, got in ((k, rk), (v, rv)):
        codes, scales = R.quantise(1, x.cpu())
        assert torch.equal(got.cpu(), R.values(1, codes, scales).bfloat16())


def test_empty(mx):
    cache = mx.MXCache.allocate(1, 2, 2, 16, 64)
    none = torch.empty((0, 2, 64), device="cuda").bfloat16()
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    mx.mx_cache_write(cache, none, none, slots)
    k, v = mx.mx_cache_read(cache, slots)
    assert k.shape == v.shape == (0, 2, 64)
