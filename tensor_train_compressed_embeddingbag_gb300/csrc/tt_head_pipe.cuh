// tt_head_pipe.cuh -- which phase of which barrier belongs to tile g of a block of
// k_head_fused.  Plain C++, so that the protocol can be walked through on the host too.
//
// A waiter tells phases apart by their parity only: while it waits for phase n of a
// barrier, phase n - 1 must be complete (or it passes at once) and phase n + 1 must not (or it
// hangs).  Two warps issue S, and two sets of dz warps take it, odd and even tiles each,
// and neither of the two waits for the other.
//   loaded   the stage holds its rows; waited for by the issuer of S
//   formed   S is there; waited for by the tile's dz warps
//   done     the stage is free: its OUT is done (log-sum-exp: its S is formed).  Waited for by
//            the TMA warp (gradients: and by the issuer of S of tile g + BUFS)
//   turned   S is read (log-sum-exp) or dz is written; waited for by the issuer of OUT
//            (log-sum-exp: of S of tile g + BUFS)
// Gradients: OUT is issued in order, which keeps a tile's phases apart by stage and by S
// buffer.  Log-sum-exp: a stage is free as soon as S is formed, so `formed` by stage can run
// a phase ahead of a slow dz warp, and by S buffer, of which there are three, odd and even
// tiles would share a barrier whose phases come in no order.  By tile modulo 2 BUFS each
// barrier has one issuer and one set, and the next phase, of tile g + 2 BUFS, needs `turned`
// of g + BUFS, which needs that of g.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define TT_HOST_DEVICE __host__ __device__
#else
#define TT_HOST_DEVICE
#endif

namespace ttemb {

struct Phase {
    uint32_t bar, n;  // barrier of its array; which phase of it, from 0
};

template <int STAGES, int BUFS, bool LSE>
struct TilePipe {
    static constexpr int kFormed = LSE ? 2 * BUFS : STAGES, kTurned = LSE ? 2 * BUFS : BUFS;  // barriers of the arrays
    TT_HOST_DEVICE static constexpr Phase loaded(uint32_t g) { return {g % STAGES, g / STAGES}; }
    TT_HOST_DEVICE static constexpr Phase formed(uint32_t g) { return {g % kFormed, g / kFormed}; }
    TT_HOST_DEVICE static constexpr Phase done(uint32_t g) { return {g % STAGES, g / STAGES}; }
    TT_HOST_DEVICE static constexpr Phase turned(uint32_t g) { return {g % kTurned, g / kTurned}; }
};

}  // namespace ttemb
