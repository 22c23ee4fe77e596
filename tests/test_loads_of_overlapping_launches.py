"""Kernels that are launched ahead begin while the launch before them still writes what they will read.  Read-only
loads (__ldg) promise that nobody does, and a compiler may move them above the wait: they are for a caller's inputs."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tensor_train_compressed_embeddingbag_gb300", "csrc")
# what the callers give: ids, rows of tables, of gradients and of x, scales of a table's rows, the losses' arrays
INPUTS = {
    "tt_lookup.cu": [r"a\.ids \+", r"unit_at<T, VEC>\(static_cast<const T\*>\(a\.in\),", r"unit_at<T, VEC>\(in,"],
    "tt_q8.cu": [r"a\.scale \+", r"unit_at<T, VEC>\(x,"],
    "tt_answers.cu": [r"a\.(logp|ref|old|adv|mask) \+", r"reinterpret_cast<const float4\*>\(p \+ i\)", r"reinterpret_cast<const unsigned\*>\(a\.mask \+ i\)"],
}


@pytest.mark.parametrize("name", sorted(INPUTS))
def test_read_only_loads_are_of_inputs(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    found = [text[m.end():m.end() + 80].split("\n")[0] for m in re.finditer(r"__ldg\(", text)]
    assert found
    for what in found:
        assert any(re.match(x, what) for x in INPUTS[name]), what
