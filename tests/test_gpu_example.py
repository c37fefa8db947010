"""The serving example runs through all of the cache's operators in both
formats (it checks its own outputs)."""
import os
import runpy
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_cached_attention_example(fmt, monkeypatch, capsys):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    monkeypatch.setattr(sys, "argv", ["cached_attention.py", "--fmt", fmt])
    runpy.run_path(os.path.join(ROOT, "examples", "cached_attention.py"), run_name="__main__")
    assert "drafted trees" in capsys.readouterr().out
