"""Rotary positions on the GPU against the formula in 64 bits: types, layouts,
odd and ragged sizes, strides, partial heads, far positions, the gradient."""
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


def frequencies(pairs, device="cuda"):
    return 10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device=device) / max(pairs, 1))


def check(y, x, pos, f, scale, layout, inverse):
    ref, mag = R.rotate(x, pos, f, scale, layout, inverse)
    # c and s, the products and the sum rounded to fp32 (4 roundings of 2^-24 cover the three), then the type's
    # rounding; dimensions that are not rotated are copied
    half_step = torch.finfo(x.dtype).eps / 2
    err = (y.double().cpu() - ref).abs()
    rot = 2 * f.numel()
    bound = half_step * ref.abs() + 4 * 2.0 ** -24 * mag * (1 + half_step) + 1e-37
    assert bool((err <= bound)[..., :rot].all()), float((err - bound).max())
    assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", [HALF, INTERLEAVED])
@pytest.mark.parametrize("tokens,heads,dim,rot", [
    (1, 1, 2, 2), (1, 32, 128, 128), (3, 5, 96, 48), (7, 3, 64, 62), (5, 2, 100, 36), (2, 3, 7, 6), (33, 1, 192, 192),
    (130, 9, 256, 128), (4, 4, 64, 0), (2, 1, 1024, 1024), (1300, 2, 64, 64), (9, 7, 80, 10)])
def test_shapes(mx, dtype, layout, tokens, heads, dim, rot):
    g = torch.Generator(device="cuda").manual_seed(tokens * 1000 + dim)
    x = torch.randn((tokens, heads, dim), generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, 1 << 20, (tokens,), generator=g, device="cuda")
    f = frequencies(rot // 2)
    for inverse in (False, True):
        check(mx.mx_rope(x, pos, f, layout=layout, scale=1.25, inverse=inverse), x, pos, f, 1.25, layout, inverse)


@pytest.mark.parametrize("layout", [HALF, INTERLEAVED])
@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 0), (2, 3), (4, 4), (8, 8)])
def test_strides_and_alignment(mx, layout, offset, pad):
    """A head range of a wider row, from an element offset, and in place."""
    tokens, heads, dim, rot = 6, 3, 64, 32
    g = torch.Generator(device="cuda").manual_seed(5)
    wide = torch.randn(tokens * (heads + 2) * (dim + pad) + 16, generator=g, device="cuda").bfloat16()
    x = wide.as_strided((tokens, heads, dim), ((heads + 2) * (dim + pad), dim + pad, 1), offset)
    pos = torch.arange(tokens, device="cuda") * 1009
    f = frequencies(rot // 2)
    y = mx.mx_rope(x, pos, f, layout=layout)
    check(y, x, pos, f, 1.0, layout, False)
    before, whole = x.clone(), wide.clone()
    out = mx.mx_rope(x, pos, f, layout=layout, dst=x)
    assert out.data_ptr() == x.data_ptr()
    assert torch.equal(x, y)
    x.copy_(before)
    assert torch.equal(wide, whole)  # nothing outside the view was touched


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_halves_that_cut_pieces_in_place(mx, dtype):
    """62 of 128 dimensions, many rows a workgroup, written over the input."""
    g = torch.Generator(device="cuda").manual_seed(62)
    x = torch.randn((37, 70, 128), generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, 1 << 17, (37,), generator=g, device="cuda")
    f = frequencies(31)
    y = mx.mx_rope(x, pos, f, scale=0.5)
    check(y, x, pos, f, 0.5, HALF, False)
    mx.mx_rope(x, pos, f, scale=0.5, dst=x)
    assert torch.equal(x, y)


def test_far_positions_keep_their_angle(mx):
    """Angles near 2^31 and beyond are reduced in 64 bits: the same bound holds."""
    x = torch.randn((4, 2, 8), device="cuda")
    pos = torch.tensor([0, 1 << 31, (1 << 40) + 7, -12345], device="cuda")
    f = torch.tensor([1.0, 0.1234567, 1e-3, 1e-9], dtype=torch.float64, device="cuda")
    check(mx.mx_rope(x, pos, f), x, pos, f, 1.0, HALF, False)


def test_inverse_is_the_gradient(mx):
    """<R x, w> differs by <dx, R^T w> for a step dx (the map is linear), and R^T R = scale^2."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x, dx, w = (torch.randn((5, 3, 96), generator=g, device="cuda") for _ in range(3))
    pos = torch.randint(0, 100000, (5,), generator=g, device="cuda")
    f = frequencies(24)
    for layout in (HALF, INTERLEAVED):
        grad = mx.mx_rope(w, pos, f, layout=layout, scale=0.75, inverse=True)
        diff = ((mx.mx_rope(x + dx, pos, f, layout=layout, scale=0.75).double() -
                 mx.mx_rope(x, pos, f, layout=layout, scale=0.75).double()) * w.double()).sum()
        want = (dx.double() * grad.double()).sum()
        # 1440 terms, each within a few roundings of 2^-24 of magnitudes of about 10
        assert abs(float(diff - want)) <= 1440 * 8 * 2.0 ** -24 * 10
        y = mx.mx_rope(mx.mx_rope(x, pos, f, layout=layout, scale=0.75), pos, f, layout=layout, scale=0.75, inverse=True)
        assert torch.allclose(y[..., :48], x[..., :48] * 0.5625, rtol=0, atol=16 * 2.0 ** -24 * float(x.abs().max()))


def test_special_values_stay_where_they_are(mx):
    """NaN and infinities reach their pair and nothing else; negative zero and lone values are copied as they are."""
    x = torch.zeros((2, 2, 16), device="cuda").bfloat16()
    x[0, 0, 1] = float("nan")
    x[0, 1, 12] = float("inf")
    x[1, 1, 13] = -0.0
    f = frequencies(4)
    y = mx.mx_rope(x, torch.tensor([3, 4], device="cuda"), f)
    bad = torch.zeros((2, 2, 16), dtype=torch.bool)
    bad[0, 0, 1] = bad[0, 0, 5] = True
    assert torch.equal(torch.isnan(y).cpu(), bad)
    assert torch.equal(y[..., 8:].view(torch.int16), x[..., 8:].view(torch.int16))


def test_empty(mx):
    x = torch.empty((0, 4, 64), device="cuda").bfloat16()
    assert mx.mx_rope(x, torch.empty(0, dtype=torch.int64, device="cuda"), frequencies(32)).shape == (0, 4, 64)
