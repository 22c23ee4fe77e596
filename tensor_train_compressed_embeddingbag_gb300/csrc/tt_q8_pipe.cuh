// tt_q8_pipe.cuh -- the rings of k_q8_scores, and what each role of a block does to them, in order.  Plain
// C++: the kernel's roles run these functions, and so does a walk through the protocol on the host.
//
//   codes     a step's table codes in shared memory.  kCfull: they are there; waited for by the set of warps that
//             turns the step's codes.  kCempty: they are in that set's registers; waited for by the codes' TMA warp
//   x         its rows of x.  kXfull: they are there; waited for by the MMA warp itself, so that no third party stands between
//             the copy and the MMAs that read it.  kXempty: the step's MMAs are done; waited for by x's TMA warp
//   tensor    its codes as f16 in tensor memory.  kTurned: they are there; waited for by the MMA warp.  kUsed: the step's
//             MMAs are done; waited for by the set of the next step in this place
//   sums      a range's accumulator, two of them.  kAccFull: its MMAs are done; waited for by the warps that write scores.
//             kAccEmpty: those have read it; waited for by the MMA warp
//
// A place of codes is let go when they are in registers, which takes more than to have issued their loads: a copy into
// the place knows of no load, and one that is still queued behind a warp's stores would read a later step's codes.
//
// A waiter tells phases apart by their parity only, so whoever waits for a phase has to have seen the
// one before.  Sets take steps in turn: with two of them a place has to belong to one set, whose waits then see
// every phase of it.  So the rings of codes and of tensor memory have even numbers of places (with three places, set 0
// could ask for step 6 while step 3, which set 1 waits for, is still on its way, and take step 0's phase for its own).  x's
// ring has one waiter, which sees every phase; its places are even in number too.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define TT_Q8_ROLE __device__ __forceinline__
#else
#define TT_Q8_ROLE inline
#endif

namespace ttemb {

template <int BN>
struct Q8Pipe {
    static constexpr int kSets = BN > 64 ? 2 : 1;
    static constexpr int kXStages = BN > 64 ? 4 : 3;
    static constexpr int kCStages = BN > 128 ? 2 : (BN > 64 ? 6 : (BN > 32 ? 3 : 5));
    static constexpr int kAStages = BN > 64 && BN <= 128 ? 4 : 2;
    static_assert(kXStages % kSets == 0 && kCStages % kSets == 0 && kAStages % kSets == 0, "a place belongs to one set");
};

enum Q8Bar { kCfull, kCempty, kXfull, kXempty, kTurned, kUsed, kAccFull, kAccEmpty };

// P: wait<B>(place, parity), false if it gave up; arrive<B>(place) of a warp, behind all that its lanes have done; commit<B>(place),
// behind all MMAs issued so far.  The rest are the role's own actions.

// load(place): the copy of step `it`'s codes.
template <int BN, class P, class Load>
TT_Q8_ROLE bool q8_feed_codes(P& p, uint32_t it, Load load) {
    constexpr uint32_t n = Q8Pipe<BN>::kCStages;
    if (!p.template wait<kCempty>(it % n, ((it / n) & 1) ^ 1)) return false;
    load(it % n);
    return true;
}

template <int BN, class P, class Load>
TT_Q8_ROLE bool q8_feed_x(P& p, uint32_t it, Load load) {
    constexpr uint32_t n = Q8Pipe<BN>::kXStages;
    if (!p.template wait<kXempty>(it % n, ((it / n) & 1) ^ 1)) return false;
    load(it % n);
    return true;
}

// Step `it` by the set whose turn it is.  read(place): issues the loads of the codes; held(): returns when they are in
// registers; put(place): writes them, as f16, to tensor memory, and returns when they are there.
template <int BN, class P, class Read, class Held, class Put>
TT_Q8_ROLE bool q8_turn(P& p, uint32_t it, Read read, Held held, Put put) {
    constexpr uint32_t c = Q8Pipe<BN>::kCStages, a = Q8Pipe<BN>::kAStages;
    if (!p.template wait<kCfull>(it % c, (it / c) & 1)) return false;
    read(it % c);
    held();
    p.template arrive<kCempty>(it % c);
    if (!p.template wait<kUsed>(it % a, ((it / a) & 1) ^ 1)) return false;
    put(it % a);
    p.template arrive<kTurned>(it % a);
    return true;
}

// The `steps` steps of accumulator number `acc`, from step `it` on.  issue(accumulator, place of x, place of codes, step of the range)
template <int BN, class P, class Issue>
TT_Q8_ROLE bool q8_multiply(P& p, uint32_t acc, uint32_t& it, int steps, Issue issue) {
    constexpr uint32_t x = Q8Pipe<BN>::kXStages, a = Q8Pipe<BN>::kAStages;
    if (!p.template wait<kAccEmpty>(acc & 1, ((acc >> 1) & 1) ^ 1)) return false;
    for (int c = 0; c < steps; ++c, ++it) {
        if (!p.template wait<kXfull>(it % x, (it / x) & 1) || !p.template wait<kTurned>(it % a, (it / a) & 1)) return false;
        issue(acc & 1, it % x, it % a, c);
        p.template commit<kUsed>(it % a);
        p.template commit<kXempty>(it % x);
    }
    p.template commit<kAccFull>(acc & 1);
    return true;
}

// read(accumulator): returns when the sums are in registers.
template <int BN, class P, class Read>
TT_Q8_ROLE bool q8_take_sums(P& p, uint32_t acc, Read read) {
    if (!p.template wait<kAccFull>(acc & 1, (acc >> 1) & 1)) return false;
    read(acc & 1);
    p.template arrive<kAccEmpty>(acc & 1);
    return true;
}

}  // namespace ttemb
