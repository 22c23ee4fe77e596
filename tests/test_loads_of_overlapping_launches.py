"""Kernels that are launched ahead begin while the launch before them still writes what they will read.  Read-only
loads (__ldg) promise that nobody does, and a compiler may move them above the wait: they are for a caller's inputs.
And a launch that ends without having waited lets the one behind it run beside the one ahead."""
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


# blocks that may end without a wait, because others of the same launch wait whatever the data are
WITHOUT = {
    "k_lookup_scatter": ["write_zeros(z, c - a.nch, gridDim.x - a.nch);"],  # beside the blocks of the chunks, one at least
    "k_lookup_few": ["zero_rows<T, VEC>(a, s.named, r0, rows);",  # only where no launch is ahead
                     "if (__syncthreads_or(earlier))"],  # the block of the id's first lookup waits
    "k_q8_few": ["if (lr >= rounds)"],  # out of a function of its own, not of the kernel
    "k_q8_scores": ["if (!lead)"],      # so too
}


def kernels_launched_ahead():
    for name in sorted(INPUTS):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        for kernel in sorted(set(re.findall(r"launch_ahead\((k_\w+)", text))):
            begin = re.search(r"__global__ void[^;{]*?\b%s\(" % kernel, text).end()
            yield kernel, text[begin:text.index("\n}\n", begin)]


def test_every_launch_ahead_waits_whatever_the_data_are():
    seen = set()
    for kernel, body in kernels_launched_ahead():
        seen.add(kernel)
        assert re.search(r"pdl_(wait|entry)\(\)", body), kernel
        last = [m.start() for m in re.finditer(r"pdl_(wait|entry)\(\)", body)][-1]
        for m in re.finditer(r"\breturn;", body[:last]):
            before = [x.split("//")[0].strip() for x in body[:m.start()].rstrip().split("\n")]
            before = [x for x in before if x and x != "{"][-1]
            if before in ("pdl_wait();", "pdl_entry();"):
                continue
            assert any(before.endswith(x) for x in WITHOUT.get(kernel, [])), (kernel, before)
    assert {"k_lookup_few", "k_lookup_scan", "k_lookup_scatter", "k_lookup_sums", "k_lookup_join", "k_answer_finish", "k_q8_few", "k_q8_scores"} <= seen
