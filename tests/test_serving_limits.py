"""Limits of the rotary, cache and attention calls: what a launch cannot hold is refused before anything is enqueued
(host only, fake addresses) or goes another way."""
import ctypes

import pytest

from test_cache_checks import A, ESHAPE, b, rope, struct  # noqa: F401 (b is a fixture)


def test_short_sequences_of_a_very_large_batch_are_divided(b):
    """A workgroup an item while that is fewer threads than a launch holds; beyond it the work is divided and needs its
    workspace."""
    keep = struct(b)
    space = b.raw().mx_cache_attention_workspace
    for batch, divided in ((1 << 20, False), ((1 << 22) - 1, False), (1 << 22, True), (1 << 24, True)):
        assert (space(ctypes.addressof(keep), 4, batch, batch, 1, 64) > 0) == divided, batch
