"""Rotary positions with several axes: the forward call and its recorded gradient against the rotation in 64 bits, keys
written to the cache bit for bit against the scalar oracle."""
import pytest
import torch

import _cacheref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from microscaling_quantize_dequantize_amd import binding
    return binding


def rotate(x, positions, axes, inv_freq, scale, layout, inverse):
    """float64 rotation, pair by pair, and sum |a c| + |b s| of each element: a pair is a head of two dimensions."""
    x = x.detach().double().cpu()
    out, mag = x.clone(), x.abs()
    n = inv_freq.numel()
    for p, (axis, f) in enumerate(zip(axes.tolist(), inv_freq.cpu())):
        at = positions[axis].cpu() if 0 <= axis < positions.shape[0] else torch.zeros(x.shape[0], dtype=torch.long)
        ia, ib = (p, p + n) if layout == 0 else (2 * p, 2 * p + 1)
        y, m = R.rotate(x[..., [ia, ib]], at, f[None], scale, 1, inverse)
        out[..., [ia, ib]], mag[..., [ia, ib]] = y, m
    return out, mag


def inputs(tokens, heads, dim, sections, dtype, seed, order="parts"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((tokens, heads, dim), generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, 1 << 16, (len(sections), tokens), generator=g, device="cuda")
    axes = [a for a, n in enumerate(sections) for _ in range(n)]
    if order == "turns":
        axes = [a for _, a in sorted((k, a) for a, n in enumerate(sections) for k in range(n))]
    pairs = len(axes)
    f = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device="cuda") / max(pairs, 1))
    return x, pos, torch.tensor(axes, dtype=torch.int32, device="cuda"), f


def check(got, want, mag, dtype):
    half_step = torch.finfo(dtype).eps / 2
    # cosine, sine, products and sum in fp32, then the type's rounding
    bound = half_step * want.abs() + 4 * 2.0 ** -24 * mag * (1 + half_step) + 1e-37
    assert bool(((got.detach().double().cpu() - want).abs() <= bound).all())


SHAPES = [(1, 1, 64, (32,)), (33, 5, 128, (16, 24, 24)), (7, 3, 96, (20, 20)), (300, 2, 64, (0, 9, 0, 5)),
          (5, 40, 128, (62, 1)), (19, 1, 10, (3, 2)), (4, 2, 64, (0,)), (1500, 4, 64, (16, 16))]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("order", ["parts", "turns"])
@pytest.mark.parametrize("tokens,heads,dim,sections", SHAPES)
def test_forward_and_inverse(mx, dtype, layout, order, tokens, heads, dim, sections):
    x, pos, axes, f = inputs(tokens, heads, dim, sections, dtype, tokens + dim, order)
    for inverse in (False, True):
        y = mx.mx_rope(x, pos, f, layout=layout, scale=1.25, inverse=inverse, axes=axes)
        check(y, *rotate(x, pos, axes, f, 1.25, layout, inverse), dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("tokens,heads,dim,sections", [(37, 5, 96, (10, 10)), (9, 3, 14, (3, 4)), (4, 2, 64, (0,))])
def test_gradient_of_a_head_range(mx, dtype, layout, tokens, heads, dim, sections):
    """Of a head range of a wider leaf: the transposed rotation there and zero beside it."""
    wide, pos, axes, f = inputs(tokens, heads + 2, dim, sections, dtype, dim)
    leaf = wide.requires_grad_()
    w = inputs(tokens, heads, dim, sections, dtype, dim + 1)[0]
    y = mx.mx_rope(leaf[:, 1:heads + 1], pos, f, layout=layout, scale=0.75, axes=axes)
    check(y, *rotate(leaf[:, 1:heads + 1], pos, axes, f, 0.75, layout, False), dtype)
    (y * w).sum().backward()
    got = leaf.grad[:, 1:heads + 1]
    check(got, *rotate(w, pos, axes, f, 0.75, layout, True), dtype)
    assert not bool(leaf.grad[:, 0].any()) and not bool(leaf.grad[:, heads + 1].any())


def test_gradient_against_differences(mx):
    """The map is linear: central differences of <y, w> along v are <R^T w, v> up to the roundings."""
    leaf, pos, axes, f = inputs(6, 5, 64, (8, 8, 8), torch.float32, 5)
    leaf.requires_grad_()
    w, v = torch.randn_like(leaf), torch.randn_like(leaf)
    (mx.mx_rope(leaf, pos, f, scale=0.5, axes=axes) * w).sum().backward()
    with torch.no_grad():
        up, down = (mx.mx_rope(leaf + s * v, pos, f, scale=0.5, axes=axes).double() for s in (1.0, -1.0))
    diff, want = ((up - down) * w.double()).sum() / 2, (leaf.grad.double() * v.double()).sum()
    # 1920 terms, each within 8 roundings of 2^-24 of magnitudes of about 20
    assert abs(float(diff - want)) <= 1920 * 8 * 2.0 ** -24 * 20


def test_gradient_of_a_shared_head(mx):
    """A head that several read, by a stride of zero: its gradient is the sum of theirs.  Four terms are added in fp32."""
    x, pos, axes, f = inputs(13, 1, 64, (16, 16), torch.float32, 4)
    leaf = x.requires_grad_()
    w = torch.randn((13, 4, 64), device="cuda")
    y = mx.mx_rope(leaf.expand(13, 4, 64), pos, f, axes=axes)
    y.backward(w)
    want, mag = rotate(w, pos, axes, f, 1.0, 0, True)
    want, mag = want.sum(1, keepdim=True), mag.sum(1, keepdim=True)
    # each term as above, and three additions of at most the sum of magnitudes
    assert bool(((leaf.grad.double().cpu() - want).abs() <= (5 + 3) * 2.0 ** -24 * mag * (1 + 2.0 ** -20)).all())


def test_second_gradient_and_sums(mx):
    """The gradient of the gradient is the rotation again; the gradient of a sum has no strides."""
    x, pos, axes, f = inputs(5, 2, 64, (16, 16), torch.float32, 3)
    x.requires_grad_()
    w = torch.randn_like(x).requires_grad_()
    g, = torch.autograd.grad(mx.mx_rope(x, pos, f, axes=axes), x, w, create_graph=True)
    v = torch.randn_like(x)
    gg, = torch.autograd.grad(g, w, v)
    check(gg, *rotate(v, pos, axes, f, 1.0, 0, False), torch.float32)
    mx.mx_rope(x, pos, f, axes=axes).sum().backward()
    check(x.grad, *rotate(torch.ones_like(x), pos, axes, f, 1.0, 0, True), torch.float32)


@pytest.mark.parametrize("layout", [0, 1])
def test_axes_that_there_are_not(mx, layout):
    """Their pairs are scaled and not turned."""
    x, pos, axes, f = inputs(11, 3, 64, (8, 8, 8), torch.float32, 7)
    axes[3], axes[10], axes[20], axes[23] = -1, 3, 1 << 30, -(1 << 31)
    y = mx.mx_rope(x, pos, f, layout=layout, scale=2.0, axes=axes)
    check(y, *rotate(x, pos, axes, f, 2.0, layout, False), torch.float32)


def test_one_axis_is_the_plain_call(mx):
    x, pos, axes, f = inputs(50, 4, 128, (40,), torch.bfloat16, 9)
    want = mx.mx_rope(x, pos[0].contiguous(), f, scale=1.5)
    assert torch.equal(mx.mx_rope(x, pos, f, scale=1.5, axes=axes), want)
    assert torch.equal(mx.mx_rope(x, pos[0].expand(3, 50), f, scale=1.5, axes=axes), want)


def test_strides_of_positions_and_in_place(mx):
    x, pos, axes, f = inputs(21, 4, 64, (10, 12, 10), torch.bfloat16, 2)
    wide = torch.zeros((3, 100), dtype=torch.int64, device="cuda")
    wide[:, 5:26] = pos
    want = mx.mx_rope(x, pos, f, axes=axes)
    assert torch.equal(mx.mx_rope(x, wide[:, 5:26], f, axes=axes), want)
    y = x.clone()
    assert mx.mx_rope(y, pos, f, dst=y, axes=axes) is y and torch.equal(y, want)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("dim,sections", [(64, (10, 12, 10)), (128, (16, 24, 24)), (96, (7, 6)), (32, (0, 1))])
def test_keys_of_the_cache(mx, fmt, layout, dim, sections):
    """Codes and scales bit for bit, except where the rotated key is within a rounding of fp64 (by way of fp32) of the
    border between two bf16 values: none of these is."""
    tokens, heads, page = 70, 3, 32
    k, pos, axes, f = inputs(tokens, heads, dim, sections, torch.bfloat16, dim + fmt)
    v = torch.randn((tokens, heads, dim), device="cuda").bfloat16()
    cache = mx.MXCache.allocate(fmt, 4, heads, page, dim)
    slots = torch.randperm(4 * page, generator=torch.Generator().manual_seed(1))[:tokens]
    mx.mx_cache_write(cache, k, v, slots.cuda(), positions=pos, inv_freq=f, layout=layout, scale=1.1, axes=axes)
    turned = rotate(k, pos, axes, f, 1.1, layout, False)[0].float().bfloat16()
    for x, codes, scales in ((turned, cache.k_codes, cache.k_scales), (v.cpu(), cache.v_codes, cache.v_scales)):
        c, s = R.quantise(fmt, x)
        assert torch.equal(codes.cpu()[slots // page, :, slots % page], c)
        assert torch.equal(scales.cpu()[slots // page, :, :, slots % page], s)


def test_gradient_beside_a_live_graph(mx):
    """Forward and backward captured while an eager graph of the same leaf lives: replays give the eager result."""
    x, pos, axes, f = inputs(64, 4, 64, (8, 12, 12), torch.float32, 8)
    w = torch.randn_like(x)
    leaf = x.requires_grad_()
    eager = mx.mx_rope(leaf, pos, f, axes=axes)
    want, = torch.autograd.grad(eager, leaf, w, retain_graph=True)

    def step(t):
        with torch.enable_grad():
            return torch.autograd.grad(mx.mx_rope(t, pos, f, axes=axes), t, w)[0]

    other = x.detach().clone().requires_grad_()  # a leaf of its own: captured work does not meet the eager graph's
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(other)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(other)
    for _ in range(3):
        held.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, want)
    again, = torch.autograd.grad(eager, leaf, w)
    assert torch.equal(again, want)
