"""The next-item example: cross entropy and distillation train a TT table that is its own
output head, and a 4-bit copy of it serves."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_learns_and_serves():
    spec = importlib.util.spec_from_file_location("next_item", os.path.join(ROOT, "examples", "next_item.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    lines = []
    got = example.main(items=1000, dim=16, rank=8, rows=256, steps=150, top=8, log=lines.append)
    assert len(lines) == 3
    for name in ("dense", "student"):
        first, last = got[name][0], sum(got[name][-10:]) / 10
        assert last < 0.8 * first, (name, first, last)
    assert got["kept"] > 0.5
