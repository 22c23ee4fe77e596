"""What the roles of the 8-bit scores' kernel hand to each other, walked through on the CPU.

csrc/tt_q8_pipe.cuh has what each role does, in order; the kernel runs these functions, and here they are compiled as
plain C++ and write down their steps.  The walk takes these programs, a role's steps in order and everything that runs
beside them (copies, loads into registers, MMAs) at any time after it was begun, in random orders, and looks at what
each of them finds: a load the codes of its step, an MMA its codes and its rows of x, the sums those of their range."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tensor_train_compressed_embeddingbag_gb300", "csrc")
BARS = ("cfull", "cempty", "xfull", "xempty", "turned", "used", "accfull", "accempty")
SHIM = r"""
#include "tt_q8_pipe.cuh"
using namespace ttemb;
static int *put, count;
static void note(int kind, int what, int place, int more) { int x[4] = {kind, what, place, more}; for (int i = 0; i < 4; ++i) put[count++] = x[i]; }
struct Written {  // 0: wait, 1: arrive, 2: commit, 3: an action of the role
    template <Q8Bar B> bool wait(uint32_t place, uint32_t parity) { note(0, B, place, parity); return true; }
    template <Q8Bar B> void arrive(uint32_t place) { note(1, B, place, 0); }
    template <Q8Bar B> void commit(uint32_t place) { note(2, B, place, 0); }
};
// role: 0 codes, 1 x, 2 mma, 3 + s set s of those that turn, 100 sums
template <int BN>
static void program(int role, const int* ranges, int n) {
    using Q = Q8Pipe<BN>;
    Written w;
    uint32_t it = 0, acc = 0;
    int steps = 0;
    for (int r = 0; r < n; ++r) steps += ranges[r];
    if (role == 0) for (; it < (uint32_t)steps; ++it) q8_feed_codes<BN>(w, it, [&](uint32_t p) { note(3, 0, p, it); });
    if (role == 1) for (; it < (uint32_t)steps; ++it) q8_feed_x<BN>(w, it, [&](uint32_t p) { note(3, 0, p, it); });
    if (role == 2)
        for (int r = 0; r < n; ++r, ++acc)
            q8_multiply<BN>(w, acc, it, ranges[r], [&](uint32_t b, uint32_t x, uint32_t a, int c) { note(3, b, x, a); note(3, c, it, 0); });
    if (role >= 3 && role < 100)
        for (int g = role - 3; g < steps; g += Q::kSets)
            q8_turn<BN>(w, g, [&](uint32_t p) { note(3, 0, p, g); }, [&]() { note(3, 1, 0, g); }, [&](uint32_t p) { note(3, 2, p, g); });
    if (role == 100) for (int r = 0; r < n; ++r) q8_take_sums<BN>(w, r, [&](uint32_t b) { note(3, 0, b, r); });
}
extern "C" int steps_of(int bn, int role, const int* ranges, int n, int* out) {
    put = out, count = 0;
    if (bn == 32) program<32>(role, ranges, n);
    if (bn == 64) program<64>(role, ranges, n);
    if (bn == 128) program<128>(role, ranges, n);
    if (bn == 192) program<192>(role, ranges, n);
    return count / 4;
}
extern "C" void shape(int bn, int* out) {
    out[0] = bn == 32 ? Q8Pipe<32>::kSets : bn == 64 ? Q8Pipe<64>::kSets : bn == 128 ? Q8Pipe<128>::kSets : Q8Pipe<192>::kSets;
}
"""
RANGES = [3, 8, 1, 5, 2]  # steps of one accumulator after the other


@pytest.fixture(scope="module")
def written(tmp_path_factory):
    d = tmp_path_factory.mktemp("roles")
    src, so = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-x", "c++", "-I" + CSRC, str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))

    def get(bn):
        """{role: [(kind, what, place, more)]}, sets"""
        sets = ctypes.c_int()
        lib.shape(bn, ctypes.byref(sets))
        out, ranges = (ctypes.c_int * 100000)(), (ctypes.c_int * len(RANGES))(*RANGES)
        programs = {}
        for name, role in [("codes", 0), ("x", 1), ("mma", 2), ("out", 100)] + [(f"set{s}", 3 + s) for s in range(sets.value)]:
            n = lib.steps_of(bn, role, ranges, len(RANGES), out)
            programs[name] = [tuple(out[4 * i:4 * i + 4]) for i in range(n)]
        return programs, sets.value
    return get


class Fault(Exception):
    pass


def walk(programs, sets, bn, rng):
    """One order of everything; raises Fault for what it finds wrong."""
    need = {"cfull": 1, "cempty": 4, "xfull": 1, "xempty": 1, "turned": 4, "used": 1, "accfull": 1, "accempty": 4 * (2 if bn > 64 else 1)}
    arrived, phase = {}, {}

    def arrive(bar, place):
        k = bar, place
        arrived[k] = arrived.get(k, 0) + 1
        if arrived[k] == need[bar]:
            arrived[k], phase[k] = 0, phase.get(k, 0) + 1

    codes, x, turned, sums = {}, {}, {}, {}
    flying, loads, mmas = [], {}, []  # copies; a warp's loads; MMAs and commits in their order
    warps = [("codes", 0), ("x", 0), ("mma", 0)] + [(f"set{s}", w) for s in range(sets) for w in range(4)] + [("out", w) for w in range(need["accempty"])]
    at = {w: 0 for w in warps}
    # a warp, or what runs beside it, may be slow for a while
    pace = {w: rng.choice([1, 1, 30]) for w in warps + ["copies", "loads", "mmas"]}
    first = [sum(RANGES[:r]) for r in range(len(RANGES))]

    def finish_load(w):
        place, step = loads.pop(w)
        if codes.get(place) != step:
            raise Fault(f"{w} loads codes of step {step} and finds those of {codes.get(place)}")

    def finish_copy(i):
        role, place, step = flying.pop(i)
        (codes if role == "codes" else x)[place] = step
        arrive("cfull" if role == "codes" else "xfull", place)

    def finish_mma():
        m = mmas.pop(0)
        if m[0] == "commit":
            arrive(*m[1:])
            return
        _, buf, px, pa, c, step = m
        for w in range(4):
            if turned.get((pa, w)) != step:
                raise Fault(f"the MMAs of step {step} find codes of step {turned.get((pa, w))}")
        if x.get(px) != step:
            raise Fault(f"the MMAs of step {step} find rows of x of step {x.get(px)}")
        sums[buf] = (sums[buf] if c else []) + [step]

    def step(w):
        role, p = w[0], programs[w[0]]
        kind, what, place, more = p[at[w]]
        if kind == 0:
            if (phase.get((BARS[what], place), 0) & 1) == more:
                return False
        elif kind == 1:
            arrive(BARS[what], place)
        elif kind == 2:
            mmas.append(("commit", BARS[what], place))
        elif role in ("codes", "x"):
            flying.append((role, place, more))
        elif role == "mma":
            c, it = p[at[w] + 1][1:3]
            mmas.append(("mma", what, place, more, c, it))
            at[w] += 1
        elif role == "out":
            want = list(range(first[more], first[more] + RANGES[more]))
            if sums.get(place) != want:
                raise Fault(f"sums of range {more} are of steps {sums.get(place)}, not {want}")
        elif what == 0:
            loads[w] = place, more
        elif what == 1:
            if w in loads:
                finish_load(w)
        else:
            if w in loads:  # the values are needed here
                finish_load(w)
            if any(m[0] == "mma" and m[3] == place for m in mmas):
                raise Fault(f"{w} writes codes of step {more} over those that MMAs still read")
            turned[place, w[1]] = more
        at[w] += 1
        return True

    while True:
        can = [w for w in warps if at[w] < len(programs[w[0]])] + ["copies"] * bool(flying) + ["loads"] * bool(loads) + ["mmas"] * bool(mmas)
        if not can:
            return
        rng.shuffle(can)
        can.sort(key=lambda w: rng.random() * pace[w])  # the slow ones seldom come first, but they do come
        for w in can:
            if w == "copies":
                finish_copy(rng.randrange(len(flying)))
            elif w == "loads":
                finish_load(rng.choice(sorted(loads)))
            elif w == "mmas":
                finish_mma()
            elif not step(w):
                continue
            break
        else:
            raise Fault("every role waits")


def found(programs, sets, bn, *what):
    """The first fault that some hundred orders show, among those of a kind if any is named."""
    for seed in range(300 if what else 100):
        try:
            walk(programs, sets, bn, random.Random(seed))
        except Fault as e:
            if not what or any(w in str(e) for w in what):
                return str(e)


@pytest.mark.parametrize("bn", [32, 64, 128, 192])
def test_every_order_finds_what_it_means(written, bn):
    programs, sets = written(bn)
    assert found(programs, sets, bn) is None


@pytest.mark.parametrize("bn", [32, 64, 128, 192])
def test_the_walk_finds_places_that_are_let_go_too_early(written, bn):
    """The walk itself: a place of codes that is free when its loads are issued, codes written without a wait for the MMAs that
    read their place, rows of x and accumulators that nobody waits for."""
    programs, sets = written(bn)

    def changed(role, change):
        return {k: change(list(v)) if k.startswith(role) else v for k, v in programs.items()}

    def early(p):  # free when the loads are issued
        return [e for e in p if e[:2] != (3, 1)]

    def without(*bars):
        return lambda p: [e for e in p if not (e[0] == 0 and BARS[e[1]] in bars)]

    assert found(changed("set", early), sets, bn, "loads codes")
    assert found(changed("set", without("used")), sets, bn, "over those that MMAs still read", "find codes")
    assert found(changed("mma", without("xfull")), sets, bn, "rows of x")
    assert found(changed("mma", without("accempty")), sets, bn, "sums of range")


@pytest.mark.parametrize("bn", [32, 64, 128, 192])
def test_the_warp_that_issues_mmas_has_waited_for_what_they_read(written, bn):
    """For the copy of the step's rows of x and for its codes, itself: what a copy brings is there for those who waited
    for the copy's own barrier."""
    p = written(bn)[0]["mma"]
    since = set()
    for i, (kind, what, place, more) in enumerate(p):
        if kind == 0:
            since.add((BARS[what], place))
        elif kind == 3 and p[i - 1][0] != 3:
            assert {("xfull", place), ("turned", more)} <= since
            since.clear()
