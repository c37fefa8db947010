"""What autograd keeps for mx_rope's gradient may come back changed (hooks on saved tensors): it is checked as the
forward call's arguments are."""
import pytest
import torch

pytestmark = pytest.mark.gpu
TOKENS, HEADS, DIM, PAIRS = 7, 3, 64, 32


@pytest.fixture(scope="module")
def mx():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from microscaling_quantize_dequantize_amd import binding
    return binding


def recorded(mx, unpack, with_axes, pack=lambda t: t):
    """A recorded call whose saved tensors go through the hooks, and the gradient that it should give."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((TOKENS, HEADS, DIM), generator=g, device="cuda", requires_grad=True)
    w = torch.randn((TOKENS, HEADS, DIM), generator=g, device="cuda")
    freq = 10000.0 ** (-torch.arange(PAIRS, dtype=torch.float64, device="cuda") / PAIRS)
    shape = (2, TOKENS) if with_axes else (TOKENS,)
    pos = torch.randint(0, 1000, shape, generator=g, device="cuda")
    axes = torch.arange(PAIRS, dtype=torch.int32, device="cuda") % 2 if with_axes else None
    with torch.autograd.graph.saved_tensors_hooks(pack, unpack):
        y = mx.mx_rope(x, pos, freq, axes=axes)
    return x, w, y, mx.mx_rope(w, pos, freq, inverse=True, axes=axes)


@pytest.mark.parametrize("with_axes", [False, True])
@pytest.mark.parametrize("which", [torch.int64, torch.float64, torch.int32])
def test_host_tensors_are_refused(mx, with_axes, which):
    if which == torch.int32 and not with_axes:
        pytest.skip("no axes")
    x, w, y, _ = recorded(mx, lambda t: t.cpu() if t.dtype == which else t, with_axes)
    with pytest.raises(TypeError, match="GPU tensor"):
        y.backward(w)
    assert x.grad is None


@pytest.mark.parametrize("with_axes", [False, True])
@pytest.mark.parametrize("change", ["stride", "length", "type"])
def test_other_forms_are_refused(mx, with_axes, change):
    def unpack(t):
        if t.dtype != torch.int64:
            return t
        if change == "type":
            return t.to(torch.int32)
        if change == "length":
            return t[..., :TOKENS - 1]
        wide = torch.zeros(t.shape + (2,), dtype=t.dtype, device="cuda")
        wide[..., 0] = t
        return wide[..., 0]

    x, w, y, _ = recorded(mx, unpack, with_axes)
    with pytest.raises(ValueError, match="positions"):
        y.backward(w)
    assert x.grad is None


@pytest.mark.parametrize("with_axes", [False, True])
@pytest.mark.parametrize("how", ["copied", "by way of the host", "rows of a wider tensor"])
def test_tensors_that_come_back_elsewhere(mx, with_axes, how):
    """The same values at another address (and, with axes, other distances of the rows) give the same gradient."""
    def unpack(t):
        if how != "rows of a wider tensor" or t.dim() == 1:
            return t.clone()
        wide = torch.full((2, TOKENS + 5), -1, dtype=t.dtype, device="cuda")
        wide[:, 2:TOKENS + 2] = t
        return wide[:, 2:TOKENS + 2]

    if how == "by way of the host":
        x, w, y, want = recorded(mx, lambda t: t.cuda(), with_axes, pack=lambda t: t.cpu())
    else:
        x, w, y, want = recorded(mx, unpack, with_axes)
    y.backward(w)
    assert torch.equal(x.grad, want)
