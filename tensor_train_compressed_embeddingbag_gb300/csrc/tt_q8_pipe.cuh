// tt_q8_pipe.cuh -- the rings of k_q8_scores: which place and which phase of its barriers belong to
// step g of a block.  Plain C++, so that the protocol can be walked through on the host too.
//
//   codes     a step's table codes in shared memory.  `cfull`: they are there; waited for by the set of warps that
//             turns the step's codes.  `cempty`: they are in that set's registers; waited for by the codes' TMA warp
//   x         its rows of x.  `xfull`: they are there; waited for by the same set, which tells the MMA warp by
//             `turned`.  `xempty`: the step's MMAs are done; waited for by x's TMA warp
//   tensor    its codes as f16 in tensor memory.  `turned`: they are there; waited for by the MMA warp.  `used`: the step's
//             MMAs are done; waited for by the set of the next step in this place
//
// A waiter tells phases apart by their parity only, so whoever waits for a phase has to have seen the
// one before.  Sets take steps in turn: with two of them a place has to belong to one set, whose waits then see
// every phase of it.  So the rings have even numbers of places (with three places for x, set 0 could ask for
// step 6 while step 3, which set 1 waits for, is still on its way, and take step 0's phase for its own).
#pragma once

#include <cstdint>

namespace ttemb {

template <int BN>
struct Q8Pipe {
    static constexpr int kSets = BN > 64 ? 2 : 1;
    static constexpr int kXStages = BN > 64 ? 4 : 3;
    static constexpr int kCStages = BN > 128 ? 2 : (BN > 64 ? 6 : (BN > 32 ? 3 : 5));
    static constexpr int kAStages = BN > 64 && BN <= 128 ? 4 : 2;
    static_assert(kXStages % kSets == 0 && kCStages % kSets == 0 && kAStages % kSets == 0, "a place belongs to one set");
};

}  // namespace ttemb
