"""The barrier protocol of the 8-bit scores' kernel, worked out on the CPU.

csrc/tt_q8_pipe.cuh has the rings; it is compiled here as plain C++.  From the steps of the roles (two
TMA warps, the sets of warps that turn codes, the MMA warp, its commits) follows what must have happened
before what.  A wait by parity is right only if the phase before the one waited for is over when the wait
begins (or it passes at once) and the phase after it cannot be over before the wait ends (or it hangs)."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tensor_train_compressed_embeddingbag_gb300", "csrc")
SHIM = r"""
#include "tt_q8_pipe.cuh"
using namespace ttemb;
template <int BN>
static void put(int* out) {
    using P = Q8Pipe<BN>;
    out[0] = P::kSets, out[1] = P::kXStages, out[2] = P::kCStages, out[3] = P::kAStages;
}
extern "C" void rings(int bn, int* out) {
    if (bn == 32) put<32>(out);
    if (bn == 64) put<64>(out);
    if (bn == 128) put<128>(out);
    if (bn == 192) put<192>(out);
}
"""


@pytest.fixture(scope="module")
def rings(tmp_path_factory):
    d = tmp_path_factory.mktemp("pipe")
    src, so = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-x", "c++", "-I" + CSRC, str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))

    def get(bn):
        out = (ctypes.c_int * 4)()
        lib.rings(bn, out)
        return tuple(out)
    return get


def roles(sets, x, c, a, steps):
    """Per role its events in order: ('wait', barrier, phase) and ('do', event); and what completes a phase."""
    done = {}  # (barrier, phase) -> the events that complete it
    programs = {"codes": [], "x": [], "mma": [], **{f"set{s}": [] for s in range(sets)}}
    for g in range(steps):
        cb, xb, ab = g % c, g % x, g % a
        if g >= c:
            programs["codes"].append(("wait", ("cempty", cb), g // c - 1))
        programs["codes"].append(("do", ("load codes", g)))
        done[("cfull", cb), g // c] = [("codes there", g)]
        if g >= x:
            programs["x"].append(("wait", ("xempty", xb), g // x - 1))
        programs["x"].append(("do", ("load x", g)))
        done[("xfull", xb), g // x] = [("x there", g)]
        p = programs[f"set{g % sets}"]
        p += [("wait", ("cfull", cb), g // c), ("do", ("read codes", g)), ("wait", ("xfull", xb), g // x)]
        done[("cempty", cb), g // c] = [("read codes", g)]
        if g >= a:
            p.append(("wait", ("used", ab), g // a - 1))
        p.append(("do", ("turned", g)))
        done[("turned", ab), g // a] = [("turned", g)]
        programs["mma"] += [("wait", ("turned", ab), g // a), ("do", ("issue", g))]
        done[("used", ab), g // a] = [("multiplied", g)]
        done[("xempty", xb), g // x] = [("multiplied", g)]
    return programs, done


def faults(sets, x, c, a, steps=26):
    programs, done = roles(sets, x, c, a, steps)
    before = {}  # event -> events that must come first, one step

    def after(event, *first):
        before.setdefault(event, set()).update(first)

    for role, program in programs.items():
        last = ("begin", role)
        for i, step in enumerate(program):
            if step[0] == "do":
                after(step[1], last)
                last = step[1]
            else:
                after(("asks", role, i), last)
                last = ("passes", role, i)
                after(last, ("asks", role, i), *done[step[1], step[2]])
    for g in range(steps):  # copies end some time after they begin, MMAs in their order
        after(("codes there", g), ("load codes", g))
        after(("x there", g), ("load x", g))
        after(("multiplied", g), ("issue", g), *([("multiplied", g - 1)] if g else []))
    known = {}

    def closure(event):
        if event not in known:
            known[event] = set()
            for e in before.get(event, ()):
                known[event] |= {e} | closure(e)
        return known[event]

    found = []
    for role, program in programs.items():
        for i, step in enumerate(program):
            if step[0] != "wait":
                continue
            barrier, phase = step[1], step[2]
            if phase and not set(done[barrier, phase - 1]) <= closure(("asks", role, i)):
                found.append((role, barrier, phase, "the phase before may be open"))
            later = done.get((barrier, phase + 1))
            if later and not any(("passes", role, i) in closure(e) for e in later):
                found.append((role, barrier, phase, "the phase after may be over"))
    return found


@pytest.mark.parametrize("bn", [32, 64, 128, 192])
def test_every_wait_is_for_the_phase_it_means(rings, bn):
    assert faults(*rings(bn)) == []


def test_odd_rings_of_two_sets_are_found():
    """The check itself: three places of x, or five of codes, between two sets."""
    assert any(f[1][0] == "xfull" for f in faults(2, 3, 4, 2))
    assert any(f[1][0] == "cfull" for f in faults(2, 4, 5, 4))
