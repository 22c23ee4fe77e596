"""The barrier protocol of the fused head kernels' tiles, walked through on the CPU.

csrc/tt_head_pipe.cuh says which phase of which barrier belongs to a tile; it is compiled
here as plain C++.  The roles of a block (TMA warp, two issuers of S, the issuer of OUT,
dz warps in two sets) are stepped in every order that the barriers allow.  A wait by
parity is right only while its barrier is in the phase waited for or has just completed
it: one phase further and the waiter hangs, one before and it does not wait."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tensor_train_compressed_embeddingbag_gb300", "csrc")
SHIM = r"""
#include "tt_head_pipe.cuh"
using namespace ttemb;
template <int S, int B, bool L>
static void put(int what, uint32_t g, uint32_t* out) {
    using P = TilePipe<S, B, L>;
    const Phase p = what == 0 ? P::loaded(g) : what == 1 ? P::formed(g) : what == 2 ? P::done(g) : P::turned(g);
    out[0] = p.bar, out[1] = p.n;
}
extern "C" void phase(int stages, int lse, int what, uint32_t g, uint32_t* out) {
    if (stages == 4) lse ? put<4, 3, true>(what, g, out) : put<4, 3, false>(what, g, out);
    else lse ? put<6, 3, true>(what, g, out) : put<6, 3, false>(what, g, out);
}
"""
LOADED, FORMED, DONE, TURNED = range(4)
BUFS = 3


@pytest.fixture(scope="module")
def phase(tmp_path_factory):
    d = tmp_path_factory.mktemp("pipe")
    src, so = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-x", "c++", "-I" + CSRC, str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))

    def get(stages, lse, what, g):
        out = (ctypes.c_uint32 * 2)()
        lib.phase(stages, int(lse), what, ctypes.c_uint32(g), out)
        return (what, out[0]), out[1]
    return get


def programs(stages, lse, phase, tiles):
    """Per role its steps: ('wait', barrier, phase) or ('arrive', barrier).  Two warps stand for each dz set."""
    at = lambda what, g: phase(stages, lse, what, g)  # noqa: E731
    wait = lambda what, g: ("wait", *at(what, g))  # noqa: E731
    arrive = lambda what, g: ("arrive", at(what, g)[0])  # noqa: E731
    tma, s, out, dz = [], [[], []], [], [[], []]
    for g in range(tiles):
        if g >= stages:
            tma.append(wait(DONE, g - stages))
        tma.append(arrive(LOADED, g))
        if g >= BUFS:
            s[g & 1].append(wait(TURNED if lse else DONE, g - BUFS))
        s[g & 1] += [wait(LOADED, g), arrive(FORMED, g)] + ([arrive(DONE, g)] if lse else [])
        dz[g & 1] += [wait(FORMED, g), arrive(TURNED, g)]
        if not lse:
            out += [wait(TURNED, g), arrive(DONE, g)]
    need = {TURNED: 2}
    return [tma, s[0], s[1]] + ([] if lse else [out]) + [dz[0], dz[0], dz[1], dz[1]], need


def walk(progs, need):
    """None, or what goes wrong in some order of the steps."""
    bars = sorted({step[1] for p in progs for step in p})
    index = {b: i for i, b in enumerate(bars)}

    def run(pcs, arrived):  # arrivals of a barrier so far; its phases completed are arrivals // need
        for r, p in enumerate(progs):
            if pcs[r] == len(p):
                continue
            step = p[pcs[r]]
            i = index[step[1]]
            if step[0] == "arrive":
                yield r, arrived[:i] + (arrived[i] + 1,) + arrived[i + 1:]
                continue
            full = arrived[i] // need.get(step[1][0], 1)
            if not step[2] <= full <= step[2] + 1:
                yield r, f"role {r} waits for phase {step[2]} of {step[1]}, which is in phase {full}"
            elif full == step[2] + 1:
                yield r, arrived

    start = ((0,) * len(progs), (0,) * len(bars))
    seen, todo = {start}, [start]
    while todo:
        pcs, arrived = todo.pop()
        moved = False
        for r, nxt in run(pcs, arrived):
            if isinstance(nxt, str):
                return nxt
            moved = True
            state = (pcs[:r] + (pcs[r] + 1,) + pcs[r + 1:], nxt)
            if state not in seen:
                seen.add(state)
                todo.append(state)
        if not moved and any(pc < len(p) for pc, p in zip(pcs, progs)):
            return f"nothing moves at {pcs}"
    return None


@pytest.mark.parametrize("stages", [4, 6])
@pytest.mark.parametrize("lse", [False, True])
def test_no_wait_misses_its_phase(phase, stages, lse):
    assert walk(*programs(stages, lse, phase, stages + 9)) is None


@pytest.mark.parametrize("formed", [4, BUFS])
def test_the_walk_finds_missed_phases(formed):
    """Log-sum-exp with `formed` by stage: a slow dz warp can be two phases behind; by S buffer: it can pass too early."""
    def of(stages, lse, what, g):
        n = {FORMED: formed, TURNED: BUFS}.get(what, stages)
        return (what, g % n), g // n
    assert "which is in phase" in walk(*programs(4, True, of, 10))
