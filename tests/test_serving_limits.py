"""Limits of the rotary, cache and attention calls: what a launch cannot hold is refused before anything is enqueued
(host only, fake addresses) or goes another way."""
import ctypes

import pytest
import torch

from test_cache_checks import A, EARG, ESHAPE, b, bf, ints, mx, rope, struct  # noqa: F401 (b and mx are fixtures)


def test_short_sequences_of_a_very_large_batch_are_divided(b):
    """A workgroup an item while that is fewer threads than a launch holds; beyond it the work is divided and needs its
    workspace."""
    keep = struct(b)
    space = b.raw().mx_cache_attention_workspace
    for batch, divided in ((1 << 20, False), ((1 << 22) - 1, False), (1 << 22, True), (1 << 24, True)):
        assert (space(ctypes.addressof(keep), 4, batch, batch, 1, 64) > 0) == divided, batch


def test_more_tokens_than_a_launch_holds(b):
    """2^32 threads and more: workgroups of 256 threads with 8 tokens (write), 16 (read), or as many as the angle table
    holds (rotary)."""
    keep = struct(b)
    c, lib = ctypes.addressof(keep), b.raw()
    for tokens in ((1 << 27) - 7, 1 << 27, (1 << 31) - 1):
        assert lib.mx_cache_write(c, A, 128, 64, A, 128, 64, A, tokens, None, None, 0, 0, 1.0) == ESHAPE
    for tokens in ((1 << 28) - 15, 1 << 28, (1 << 31) - 1):
        assert lib.mx_cache_read(c, A, tokens, A, A) == ESHAPE
    for rot, tokens in ((4096, 1 << 24), (4096, (1 << 31) - 1), (64, (1 << 30) - 63), (34, (1 << 31) - 1)):
        assert rope(b, dim=4096, rot=rot, tokens=tokens) == ESHAPE


def test_scale_whose_factor_overflows(b):
    """The kernels multiply scores by scale * log2(e), which has to be finite too: zero scores would become NaN."""
    keep = struct(b)
    for scale in (2.36e38, 3.4e38):
        assert b.raw().mx_cache_attention(ctypes.addressof(keep), A, 256, 64, 4, A, A, 2, A, 4, 4, 2, 1, 64, None, 0,
                                          scale, A, A, 1 << 30) == EARG


def test_cache_without_heads_is_refused(mx):
    with pytest.raises(ValueError, match="heads"):
        mx.MXCache.allocate(1, 2, 0, 16, 64, device="cpu")
    with pytest.raises(ValueError, match="heads"):
        mx.MXCache.allocate(1, 1, 65536, 16, 32, device="cpu")


@pytest.mark.parametrize("dim", [32, 160, 224])
def test_heads_that_attention_does_not_take(mx, dim):
    """A cache may have them (they are written and read); attention says which it takes."""
    cache = mx.MXCache.allocate(0, 2, 1, 16, dim, device="cpu")
    i32 = torch.int32
    with pytest.raises(ValueError, match="64, 96, 128, 192, 256"):
        mx.mx_cache_attention(cache, bf(2, 1, dim), ints(3, dtype=i32), ints(2, dtype=i32), ints(2, 2, dtype=i32),
                              max_q=1, max_kv=20)


def test_stream_without_the_private_call(b, monkeypatch):
    """A torch that lacks the quick way to the stream's handle is served by the public one."""
    import importlib.util
    import types
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: types.SimpleNamespace(cuda_stream=1000 + device))
    spec = importlib.util.spec_from_file_location("binding_without", b.__file__)
    again = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(again)
    try:
        again._stream()
        assert again.raw().mx_get_stream() == 1003
    finally:
        again.raw().mx_set_stream(None)
