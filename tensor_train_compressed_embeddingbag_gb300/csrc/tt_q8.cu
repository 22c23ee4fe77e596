// tt_q8.cu -- scores against a table held in 8-bit integers:
//
//   out[m, v] = xscale[m] scale[v] sum_d xcode[m, d] code[v, d]
//
// The rows of x are quantized first (k_q8_rows), then multiplied (k_q8_scores).
//
// This part's tensor cores have no fast path for integers.  But an 8-bit code is an f16 value, the
// product of two is below 2^14, and a sum of 1,024 of them at most 2^24: the f16 path with fp32
// accumulation gives the exact integer for up to 1,024 columns.  Longer rows are added up in such
// ranges as int32 in registers.
//
// The table stays in 8 bits until it is on the chip: TMA brings 128 rows x 128 columns of codes, one or two
// sets of four warps turn them into f16 (one byte permutation puts a code, made unsigned, into the mantissa of 1024; one
// packed subtraction leaves it) and write them to tensor memory, from where the MMA takes its A
// operand.  The codes of x, few against the table's, are f16 in memory from the start and come by TMA as
// the B operand.  So the accumulator's rows are table rows and its columns rows of x, and a
// warp that stores 32 lanes of a column writes 128 consecutive bytes of a row of scores.
//
// Measured, rows of x by the table, quantizing included: 2048 x 131072 x 2048 722 to 739 us (1,490 to 1,520 TFLOP/s), 192 x 131072
// x 4096 168 (1,227 TFLOP/s), 128 x 131072 x 4096 127 (4.8 TB/s), 33 x 131072 x 4096 100 (5.5 TB/s), 1 x 131072 x 4096 97 (5.5 TB/s),
// 33 x 50001 x 1000 25.
#include <algorithm>

#include "tt_q8_pipe.cuh"
#include "tt_units.cuh"

namespace ttemb {

constexpr int kQ8K = 128;         // columns of a step
constexpr int kQ8Range = 1024;    // columns that an accumulator takes (a multiple of kQ8K)
constexpr int kQ8ACols = kQ8K / 2;  // tensor-memory columns of a step's codes

// Warps: 0 rows of x, 1 MMA, 2 tensor memory, 3 codes; then kSets x 4 codes to f16, kParts x 4 scores out (a part
// of the columns each).
//
// What bounds a narrow tile is the warp that issues the MMAs: a step costs it some 190 cycles of waiting, 60 for each
// of the eight MMAs and 90 for each commit, whatever their width (clock stamps, taken before it waited for the rows of x itself).  So up to 64 rows of x two blocks share a
// multiprocessor, each with half of its shared and tensor memory.
template <int BN>
struct Q8Shape : Q8Pipe<BN> {
    using Q8Pipe<BN>::kSets;
    using Q8Pipe<BN>::kXStages;
    using Q8Pipe<BN>::kCStages;
    using Q8Pipe<BN>::kAStages;
    static constexpr int kBlocks = BN > 64 ? 1 : 2;  // of a multiprocessor
    static constexpr int kParts = BN > 64 ? 2 : 1, kCols = BN / kParts;
    static constexpr int kThreads = (4 + 4 * kSets + 4 * kParts) * 32;
    // a step's codes leave shared memory early, its rows of x when its MMAs are done: a ring for each
    static constexpr uint32_t kC = 128 * kQ8K, kX = BN * kQ8K * 2;
    static constexpr size_t kSmem = (size_t)kXStages * kX + (size_t)kCStages * kC + 1024;
    static constexpr int kTmem = 512 / kBlocks;        // columns
    static constexpr int kACol = 2 * BN;               // behind the two accumulators: kAStages steps
    // 192 columns take 96 sums a thread in the last eight warps: registers go there from the others
    static constexpr bool kShift = BN > 128;
    static_assert(kACol + kAStages * kQ8ACols <= kTmem && kBlocks * (kSmem + 2048) <= 228 * 1024, "tensor and shared memory");
};

struct Q8Args {
    int64_t M, V;
    int mtiles;
    int64_t units;     // table tiles x mtiles
    int chunks;        // of kQ8K columns
    const float* xscale;
    const float* scale;
    float* out;
    uint64_t wait_ns;
    int* err;
};

// One box of a 2-D tensor map into shared memory.
__device__ __forceinline__ void tma_load2(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(x),
        "r"(y), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// Four 8-bit codes as two pairs of f16.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u;  // code + 128
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);  // 1024 + code + 128
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
}

// Registers of a thread from here on, for all four warps of a group.  A launch of 640 threads has 640 x 96 of them; the
// groups' shares add up to that: 48 + 2 x 88 + 2 x 128 = 5 x 96.
constexpr int kQ8Regs = 96, kQ8RegsFeed = 48, kQ8RegsTurn = 88, kQ8RegsOut = 128;
static_assert(kQ8RegsFeed + 2 * kQ8RegsTurn + 2 * kQ8RegsOut <= 5 * kQ8Regs, "more would never be there");
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// The block's barriers, and how the roles of tt_q8_pipe.cuh use them.
template <int BN>
struct Q8Barriers {
    using S = Q8Pipe<BN>;
    uint64_t cfull[S::kCStages], cempty[S::kCStages], xfull[S::kXStages], xempty[S::kXStages];
    uint64_t turned[S::kAStages], used[S::kAStages], accfull[2], accempty[2], drain;
    template <Q8Bar B>
    __device__ __forceinline__ uint64_t* at(uint32_t place) {
        if constexpr (B == kCfull) return &cfull[place];
        if constexpr (B == kCempty) return &cempty[place];
        if constexpr (B == kXfull) return &xfull[place];
        if constexpr (B == kXempty) return &xempty[place];
        if constexpr (B == kTurned) return &turned[place];
        if constexpr (B == kUsed) return &used[place];
        if constexpr (B == kAccFull) return &accfull[place];
        if constexpr (B == kAccEmpty) return &accempty[place];
    }
};
template <int BN>
struct Q8Roles {
    Q8Barriers<BN>& bars;
    uint64_t wait_ns;
    volatile int* gave_up;
    bool lead;
    template <Q8Bar B>
    __device__ __forceinline__ bool wait(uint32_t place, uint32_t parity) {
        return head_wait(bars.template at<B>(place), parity, wait_ns, gave_up);
    }
    template <Q8Bar B>
    __device__ __forceinline__ void arrive(uint32_t place) {
        __syncwarp();
        if (lead) mbar_arrive(bars.template at<B>(place));
    }
    template <Q8Bar B>
    __device__ __forceinline__ void commit(uint32_t place) {
        mma_commit(bars.template at<B>(place), lead);
    }
};

// A unit is 128 table rows x BN rows of x; the tiles of x go fastest, so blocks that run together
// share table rows.
template <int BN>
__global__ void __launch_bounds__(Q8Shape<BN>::kThreads, Q8Shape<BN>::kBlocks)
    k_q8_scores(const __grid_constant__ CUtensorMap map_codes, const __grid_constant__ CUtensorMap map_x, const __grid_constant__ Q8Args a) {
    using S = Q8Shape<BN>;
    constexpr int kCols = S::kCols;      // columns of an epilogue warp
    constexpr int kOutWarp = 4 + 4 * S::kSets;
    constexpr int kRangeSteps = kQ8Range / kQ8K;
    extern __shared__ uint8_t raw[];
    __shared__ Q8Barriers<BN> bars;
    __shared__ uint32_t tmem_slot;
    __shared__ int gave_up_s;
    __shared__ volatile uint32_t taken[4 * S::kSets][32];  // never read
    volatile int* gave_up = &gave_up_s;
    const uint32_t xbase = (smem_addr(raw) + 1023u) & ~1023u, cbase = xbase + S::kXStages * S::kX;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const bool lead = lane == 0;
    Q8Roles<BN> roles{bars, a.wait_ns, gave_up, lead};

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kCStages; ++i) {
            mbar_init(&bars.cfull[i], 1);
            mbar_init(&bars.cempty[i], 4);  // the warps of a set: their codes are in registers
        }
        for (int i = 0; i < S::kXStages; ++i) {
            mbar_init(&bars.xfull[i], 1);
            mbar_init(&bars.xempty[i], 1);
        }
        for (int i = 0; i < S::kAStages; ++i) {
            mbar_init(&bars.turned[i], 4);  // a set's codes are in tensor memory
            mbar_init(&bars.used[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.accfull[i], 1);
            mbar_init(&bars.accempty[i], 4 * S::kParts);
        }
        mbar_init(&bars.drain, 1);
        gave_up_s = 0;
    }
    if (warp == 2) tc_alloc(&tmem_slot, S::kTmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // one value for the warp, known to the compiler to be so: the MMAs' addresses stay in uniform registers
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
    // steps of this block's units, one behind the other
    const int64_t mine = a.units > blockIdx.x ? (a.units - 1 - blockIdx.x) / gridDim.x + 1 : 0, total = mine * a.chunks;
    uint32_t it = 0;   // steps fed or multiplied
    uint32_t acc = 0;  // accumulators filled or read
    bool ok = true;

    if (warp < 4) {
        if (S::kShift) fewer_registers<kQ8RegsFeed>();
        if (warp == 0 || warp == 3) {
            const bool x = warp == 0;
            if (x) pdl_wait();  // x is being quantized; the codes need not wait for that
            for (int64_t u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
                const int v = (int)(u / a.mtiles), m = (int)(u - (int64_t)v * a.mtiles);
                for (int c = 0; c < a.chunks; ++c, ++it) {
                    if (x) {
                        ok = q8_feed_x<BN>(roles, it, [&](uint32_t st) {
                            if (!lead) return;
                            const uint32_t to = xbase + st * S::kX;
                            bulk_expect(&bars.xfull[st], S::kX);
                            tma_load2(to, &map_x, c * kQ8K, m * BN, &bars.xfull[st]);
                            tma_load2(to + S::kX / 2, &map_x, c * kQ8K + 64, m * BN, &bars.xfull[st]);
                        });
                    } else {
                        ok = q8_feed_codes<BN>(roles, it, [&](uint32_t st) {
                            if (!lead) return;
                            tc_fence_smem();  // the set's loads from this place before the copy into it
                            bulk_expect(&bars.cfull[st], S::kC);
                            tma_load2(cbase + st * S::kC, &map_codes, c * kQ8K, v * 128, &bars.cfull[st]);
                        });
                    }
                    if (!ok) break;
                    __syncwarp();
                }
            }
        } else if (warp == 1) {
            const uint32_t idesc = idesc_f16(128, BN, 0, false, false);
            const uint32_t db0 = desc_lo(xbase, kNoLbo);
            for (int64_t i = 0; ok && i < mine; ++i) {
                for (int r0 = 0; ok && r0 < a.chunks; r0 += kRangeSteps, ++acc) {
                    ok = q8_multiply<BN>(roles, acc, it, min(kRangeSteps, a.chunks - r0), [&](uint32_t buf, uint32_t st, uint32_t ta, int c) {
                        tc_fence_after();
                        const uint32_t d = tmem + buf * BN, pa = tmem + S::kACol + ta * kQ8ACols, db = db0 + st * (S::kX >> 4);
#pragma unroll
                        for (int k = 0; k < kQ8K / 16; ++k)
                            mma_f16_ta(d, pa + k * 8, db + (k >= 4 ? (S::kX / 2) >> 4 : 0) + (k & 3) * (32 >> 4), idesc, c > 0 || k > 0, lead);
                    });
                }
            }
        }
    } else if (warp < kOutWarp) {
        if (S::kShift) fewer_registers<kQ8RegsTurn>();
        const uint32_t set = (warp - 4) >> 2;
        const int quad = warp & 3, r = quad * 32 + lane;
        const uint32_t to = tmem + ((uint32_t)(quad * 32) << 16) + S::kACol;
        for (int64_t i = set; ok && i < total; i += S::kSets) {
            uint4 w[8];
            uint32_t q[4][16];
            auto turn = [&](int h) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint4 y = w[h * 2 + x];
                    codes_to_f16(y.x, q[h][x * 8], q[h][x * 8 + 1]);
                    codes_to_f16(y.y, q[h][x * 8 + 2], q[h][x * 8 + 3]);
                    codes_to_f16(y.z, q[h][x * 8 + 4], q[h][x * 8 + 5]);
                    codes_to_f16(y.w, q[h][x * 8 + 6], q[h][x * 8 + 7]);
                }
            };
            // where there are registers, the codes are f16 before the MMAs that still read this place are done
            constexpr bool kEarly = S::kBlocks == 1;
            ok = q8_turn<BN>(
                roles, (uint32_t)i,
                [&](uint32_t cs) {
                    const uint32_t row = cbase + cs * S::kC + r * 128;
#pragma unroll
                    for (int x = 0; x < 8; ++x) w[x] = lds16(row + ((x ^ (r & 7)) << 4));  // 128-byte swizzle
                    if (kEarly)
#pragma unroll
                        for (int h = 0; h < 4; ++h) turn(h);
                },
                // A store of a word that takes one of each load: it waits for all of them, and the arrival, behind it, for it.  (Writing
                // the codes to tensor memory first would do too: 2048 x 131072 x 2048 830 us, 723 this way.)
                [&]() { taken[warp - 4][lane] = w[0].x ^ w[1].x ^ w[2].x ^ w[3].x ^ w[4].x ^ w[5].x ^ w[6].x ^ w[7].x; },
                [&](uint32_t ta) {
                    tc_fence_after();
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        if (!kEarly) turn(h);
                        tm_st16(to + ta * kQ8ACols + h * 16, q[h]);
                    }
                    tm_wait_st();
                    tc_fence_before();
                });
        }
    } else {
        if (S::kShift) more_registers<kQ8RegsOut>();
        pdl_wait();  // the scales of x
        const int part = (warp - kOutWarp) >> 2, quad = warp & 3;
        for (int64_t u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
            const int vt = (int)(u / a.mtiles), mt = (int)(u - (int64_t)vt * a.mtiles);
            const int64_t v = (int64_t)vt * 128 + quad * 32 + lane, m0 = (int64_t)mt * BN + part * kCols;
            const int rows = (int)min((int64_t)kCols, a.M - m0);  // may be below 1
            // the scales are on their way while the sums are formed; a column's is in one lane and goes to all
            const float s = v < a.V ? __ldg(a.scale + v) : 0.f;
            float xs[(kCols + 31) / 32];
#pragma unroll
            for (int h = 0; h < kCols; h += 32) xs[h / 32] = h + lane < rows ? a.xscale[m0 + h + lane] : 0.f;
            int sum[kCols];
#pragma unroll 1
            for (int r0 = 0; ok && r0 < a.chunks; r0 += kRangeSteps, ++acc)
                ok = q8_take_sums<BN>(roles, acc, [&](uint32_t buf) {
                    tc_fence_after();
                    const uint32_t t0 = tmem + buf * BN + ((uint32_t)(quad * 32) << 16) + part * kCols;
#pragma unroll
                    for (int h = 0; h < kCols; h += 16) {
                        float x[16];
                        tm_read16(t0 + h, x);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const int y = __float2int_rn(x[j]);
                            sum[h + j] = r0 == 0 ? y : sum[h + j] + y;
                        }
                    }
                    tc_fence_before();
                });
            if (!ok) break;
            float* o = a.out + m0 * a.V + v;
#pragma unroll
            for (int j = 0; j < kCols; ++j) {
                const float f = __shfl_sync(0xffffffffu, xs[j / 32], j & 31);
                if (j < rows && v < a.V) *o = (float)sum[j] * (f * s);
                o += a.V;
            }
        }
    }
    if (!ok && lead) {
        *gave_up = 1;
        if (a.err) atomicOr(a.err, kErrTimeout);
    }
    __syncwarp();
    __syncthreads();
    if (*gave_up) {  // no copy and no MMA may still be running when the block ends
        if (threadIdx.x == 0)
            for (uint32_t i = it > S::kXStages ? it - S::kXStages : 0; i < it; ++i) head_drain(&bars.xfull[i % S::kXStages], (i / S::kXStages) & 1);
        if (threadIdx.x == 96)
            for (uint32_t i = it > S::kCStages ? it - S::kCStages : 0; i < it; ++i) head_drain(&bars.cfull[i % S::kCStages], (i / S::kCStages) & 1);
        if (threadIdx.x == 32) {
            mma_commit(&bars.drain, true);
            head_drain(&bars.drain, 0);
        }
        __syncwarp();
        __syncthreads();
    }
    tc_fence_after();
    if (warp == 2) tc_dealloc(tmem, S::kTmem);
}

// ---------------------------------------------------------------- few rows
//
// Few rows of x are a stream: the table's bytes are the floor.  Here a tile's way through shared
// and tensor memory would cost more than its bytes (a step of the kernel above takes its issuing warp some
// 700 cycles, whatever it multiplies), so the codes go from global memory to registers, 16 bytes of
// a row to a thread, become f16 there and are multiplied by the warp-level tensor cores
// (mma.sync.m16n8k16: 16 table rows x 8 rows of x).  The order of k is free as long as both operands use the
// same: a thread's 16 columns of a row are the k of four MMAs, and x lies in memory in the order in which the
// fragments want it.
constexpr int kFewThreads = 256, kFewWarps8 = kFewThreads / 32;
constexpr int kFewTile = 32;   // table rows of a warp
constexpr int kFewK = 64;      // columns of a step

// Where element d of row m is: [step][tile of 8 rows][half of a thread's 16 columns][row, quarter of 64 columns][8].
__host__ __device__ __forceinline__ int64_t few_at(int64_t m, int d, int ntiles) {
    return ((((int64_t)(d >> 6) * ntiles + (m >> 3)) * 2 + ((d >> 3) & 1)) * 32 + (m & 7) * 4 + ((d >> 4) & 3)) * 8 + (d & 7);
}

__device__ __forceinline__ void mma_codes(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct FewArgs8 {
    const int8_t* codes;
    int64_t pitch, V;
    const float* scale;
    const uint4* x;        // few_at
    const float* xscale;
    int M, steps;          // of kFewK columns
    int ksplit;            // warps that share the columns of a table tile
    float* out;
};

// LONG: rows of the table are long: registers hold loads in flight; else a tile is soon over, and they hold the
// scales of the next one (1 x 131072 x 4096: 92 us, 100 the other way; 1 x 1,000,000 x 64: 26 and 19).
template <int NT, bool LONG>
__global__ void __launch_bounds__(kFewThreads, 2) k_q8_few(const __grid_constant__ FewArgs8 a) {
    constexpr int kAhead = LONG ? 4 : 2;  // steps in flight
    __shared__ int red[kFewWarps8][NT * 8 * kFewTile];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int per = kFewWarps8 / a.ksplit, sub = warp / a.ksplit, ks = warp - sub * a.ksplit;
    const int jb = a.steps * ks / a.ksplit, je = a.steps * (ks + 1) / a.ksplit;
    const int64_t tiles = (a.V + kFewTile - 1) / kFewTile, rounds = (tiles + per - 1) / per;
    // the next step to load: four table rows per thread (rows past V read row V - 1)
    int64_t lr = blockIdx.x;
    int lj = jb;
    const int8_t* row[4];
    auto at_tile = [&]() {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t v = (lr * per + sub) * kFewTile + r * 8 + g;
            row[r] = a.codes + (v < a.V ? v : a.V - 1) * a.pitch;
        }
    };
    at_tile();
    uint4 q[kAhead][4];
    auto load = [&](uint4 (&w)[4]) {
        if (lr >= rounds) return;
        const int64_t d = (int64_t)lj * kFewK + t * 16;
#pragma unroll
        for (int r = 0; r < 4; ++r) w[r] = __ldcs(reinterpret_cast<const uint4*>(row[r] + (d < a.pitch ? d : 0)));  // past the end x is 0
        if (++lj == je) {
            lj = jb;
            lr += gridDim.x;
            if (lr < rounds) at_tile();
        }
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(q[i]);
    float s_now[4], s_next[4];  // not LONG: the scales of this tile's rows and of the next one's (with columns shared, the joining lanes read them)
    auto scales = [&](int64_t round, float (&s)[4]) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t v = (round * per + sub) * kFewTile + r * 8 + g;
            s[r] = a.ksplit == 1 && v < a.V ? __ldg(a.scale + v) : 0.f;
        }
    };
    if (!LONG) scales(blockIdx.x, s_now);
    pdl_wait();  // x, and its scales
    float xs[NT][2];  // (LONG reads them again: no registers)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) xs[n][e] = n * 8 + 2 * t + e < a.M ? a.xscale[n * 8 + 2 * t + e] : 0.f;
    int sum[2][NT][4];
    float acc[2][NT][4];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sum[r][n][e] = 0;
                acc[r][n][e] = 0.f;
            }
    int in_range = 0;  // steps in acc: at most 1,024 columns, whose sums are exact
    auto settle = [&]() {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sum[r][n][e] += __float2int_rn(acc[r][n][e]);
                    acc[r][n][e] = 0.f;
                }
        in_range = 0;
    };
    int64_t rd = blockIdx.x;
    int j = jb;
    while (rd < rounds) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (rd >= rounds) break;
            if (!LONG && j == jb) scales(rd + gridDim.x, s_next);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint4 x[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) x[n] = a.x[((int64_t)(j * NT + n) * 2 + h) * 32 + lane];
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    uint32_t lo[4], hi[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const uint32_t c = h == 0 ? (w == 0 ? q[i][r].x : q[i][r].y) : (w == 0 ? q[i][r].z : q[i][r].w);
                        codes_to_f16(c, lo[r], hi[r]);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint32_t b0 = w == 0 ? x[n].x : x[n].z, b1 = w == 0 ? x[n].y : x[n].w;
                        mma_codes(acc[0][n], lo[0], lo[1], hi[0], hi[1], b0, b1);
                        mma_codes(acc[1][n], lo[2], lo[3], hi[2], hi[3], b0, b1);
                    }
                }
            }
            load(q[i]);
            if (++in_range == kQ8Range / kFewK) settle();
            if (++j < je) continue;
            settle();
            // element (row, m) of n tile n: row r * 16 + (e >> 1) * 8 + g, m = n * 8 + 2 t + (e & 1)
            const int64_t v0 = (rd * per + sub) * kFewTile;
            if (a.ksplit == 1) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int64_t v = v0 + r * 8 + g;
                    if (v >= a.V) continue;
                    const float s = LONG ? __ldg(a.scale + v) : s_now[r];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int m = n * 8 + 2 * t + e;
                            if (m < a.M) a.out[(int64_t)m * a.V + v] = (float)sum[r >> 1][n][(r & 1) * 2 + e] * ((LONG ? a.xscale[m] : xs[n][e]) * s);
                        }
                }
            } else {  // joined with the other warps of the tile
                __syncthreads();
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int e = 0; e < 4; ++e) red[warp][(n * 8 + 2 * t + (e & 1)) * kFewTile + r * 16 + (e >> 1) * 8 + g] = sum[r][n][e];
                __syncthreads();
                const int64_t v = v0 + lane;
                for (int m = ks; m < a.M; m += a.ksplit) {
                    if (v >= a.V) continue;
                    int s = 0;
                    for (int k = 0; k < a.ksplit; ++k) s += red[sub * a.ksplit + k][m * kFewTile + lane];
                    a.out[(int64_t)m * a.V + v] = (float)s * (a.xscale[m] * __ldg(a.scale + v));
                }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[r][n][e] = 0;
            if (!LONG)
#pragma unroll
                for (int r = 0; r < 4; ++r) s_now[r] = s_next[r];
            j = jb;
            rd += gridDim.x;
        }
    }
}

// 127 x / top rounded to nearest, ties to even, as if the quotient were exact: the fp32 product by
// 127 / top is off by less than 2^-16, so only next to a tie the two are compared exactly (a
// product of 24 and 8 bits fits a double).
__device__ __forceinline__ float code_of(float x, float top, float inv) {
    const float q = x * inv, k = rintf(q);
    if (fabsf(fabsf(q - k) - 0.5f) > 0.0001f) return k;
    const float lo = floorf(q);  // the tie is at lo + 1/2
    const double d = 254.0 * (double)x - (2.0 * (double)lo + 1.0) * (double)top;
    if (d != 0.0) return d > 0.0 ? lo + 1.f : lo;
    return fmodf(lo, 2.f) == 0.f ? lo : lo + 1.f;
}

// Codes of the rows of a matrix: int8 (out8) or as f16 values (out16), columns up to `pitch` with 0;
// ntiles > 0: f16 in the order of few_at.
// `lanes` threads to a row, which keep kQ8Held units each in registers and read what is beyond twice.
constexpr int kQ8Held = 4;
template <class T, int VEC>
__global__ void __launch_bounds__(256) k_q8_rows(const T* x, int64_t ld, int64_t rows, int D, int lanes, int8_t* out8, __half* out16, int64_t pitch,
                                                 int ntiles, float* scales) {
    __shared__ uint32_t top_s[8];
    const int per = 256 / lanes, sub = threadIdx.x / lanes, lane = threadIdx.x & (lanes - 1), units = D / VEC;
    const int64_t blocks = (rows + per - 1) / per;
    pdl_launch_dependents();
    for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        const int64_t r = b * per + sub;
        const bool live = r < rows;
        Raw<T, VEC> held[kQ8Held];
        uint32_t most = 0;  // bits of the largest magnitude; infinities and NaN are above all others
        auto take = [&](const Raw<T, VEC>& w) {
            float y[VEC];
            unpack<T, VEC>(w, y);
#pragma unroll
            for (int j = 0; j < VEC; ++j) most = max(most, __float_as_uint(y[j]) & 0x7FFFFFFFu);
        };
        if (live) {
#pragma unroll
            for (int i = 0; i < kQ8Held; ++i)
                held[i] = lane + i * lanes < units ? __ldg(unit_at<T, VEC>(x, r, ld, lane + i * lanes)) : raw_zero<T, VEC>();
#pragma unroll
            for (int i = 0; i < kQ8Held; ++i) take(held[i]);
#pragma unroll 4
            for (int u = lane + kQ8Held * lanes; u < units; u += lanes) take(__ldg(unit_at<T, VEC>(x, r, ld, u)));
        }
        for (int o = min(lanes, 32) / 2; o; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        if (lanes > 32) {
            if ((threadIdx.x & 31) == 0) top_s[threadIdx.x >> 5] = most;
            __syncthreads();
            for (int w = sub * (lanes / 32); w < (sub + 1) * (lanes / 32); ++w) most = max(most, top_s[w]);
            __syncthreads();
        }
        if (!live) continue;
        const float top = __uint_as_float(most);
        if (lane == 0) scales[r] = most > 0x7F800000u ? __int_as_float(0x7FC00000) : __fdiv_rn(top, 127.f);
        const bool finite = most < 0x7F800000u && most > 0;
        // 127 / top is infinite below 2^-120: both times 2^100, which changes no quotient
        const float up = finite && most < 0x03800000u ? 0x1p100f : 1.f, big = top * up, inv = 127.f / big;
        auto put = [&](int u, const Raw<T, VEC>& w) {
            float y[VEC];
            unpack<T, VEC>(w, y);
            float k[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                k[j] = finite ? code_of(y[j] * up, big, inv) : 0.f;
                if (most == 0x7F800000u) k[j] = fabsf(y[j]) == INFINITY ? copysignf(1.f, y[j]) : 0.f;
            }
            if constexpr (VEC == 1) {
                if (out8)
                    out8[r * pitch + u] = (int8_t)(int)k[0];
                else
                    out16[ntiles ? few_at(r, u, ntiles) : r * pitch + u] = __float2half_rn(k[0]);
            } else if (out8) {
#pragma unroll
                for (int j = 0; j < VEC; j += 4) {
                    const uint32_t q = ((uint32_t)(int)k[j] & 255u) | ((uint32_t)(int)k[j + 1] & 255u) << 8 | ((uint32_t)(int)k[j + 2] & 255u) << 16 |
                                       (uint32_t)(int)k[j + 3] << 24;
                    *reinterpret_cast<uint32_t*>(out8 + r * pitch + (int64_t)u * VEC + j) = q;
                }
            } else {
#pragma unroll
                for (int j = 0; j < VEC; j += 4)
                    *reinterpret_cast<uint2*>(out16 + (ntiles ? few_at(r, u * VEC + j, ntiles) : r * pitch + (int64_t)u * VEC + j)) =
                        make_uint2(pack16(k[j], k[j + 1], 0), pack16(k[j + 2], k[j + 3], 0));
            }
        };
#pragma unroll
        for (int i = 0; i < kQ8Held; ++i)
            if (lane + i * lanes < units) put(lane + i * lanes, held[i]);
        for (int u = lane + kQ8Held * lanes; u < units; u += lanes) put(u, __ldg(unit_at<T, VEC>(x, r, ld, u)));
        for (int64_t d = D + lane; d < pitch; d += lanes) {
            if (out8)
                out8[r * pitch + d] = 0;
            else
                out16[ntiles ? few_at(r, (int)d, ntiles) : r * pitch + d] = __float2half_rn(0.f);
        }
    }
}

namespace {

tt_status q8_sizes(int64_t rows, int64_t dim, int dtype) {
    if (dtype != TT_F32 && dtype != TT_BF16 && dtype != TT_F16) return TT_ERR_ARG;
    if (rows < 0 || rows > TT_HEAD_MAX_VOCAB || dim < 1 || dim > TT_HEAD_MAX_DIM) return TT_ERR_SHAPE;
    return TT_OK;
}

int64_t x_pitch(int64_t dim) { return (dim + 7) / 8 * 8; }
int64_t code_pitch(int64_t dim) { return (dim + 15) / 16 * 16; }

int64_t few_pitch(int64_t dim) { return (dim + kFewK - 1) / kFewK * kFewK; }
// Tiles of 8 rows, 0: not few.  Up to 8 rows a stream is the fastest everywhere (8 x 131072 x 4096: 102 us, 106 the
// other way); 9 to 16 cost it twice the multiplications, which it keeps up with only where rows of the table are short and the
// other kernel has nothing to overlap its tiles' fill and drain with (16 rows: 1,000,000 x 64 38 us, 42 the other way; 131072 x 4096 128, 99).
int few_tiles(int64_t rows, int64_t dim) { return rows <= 8 ? 1 : (rows <= 16 && dim <= 256 ? 2 : 0); }

struct Q8Space {
    __half* x;
    float* xscale;
    size_t bytes;
};
Q8Space q8_space(int64_t rows, int64_t dim, void* ws) {
    const int nt = few_tiles(rows, dim);
    const size_t codes = ((size_t)(nt ? (int64_t)nt * 8 * few_pitch(dim) : rows * x_pitch(dim)) * 2 + 255) / 256 * 256;
    uint8_t* p = static_cast<uint8_t*>(ws);
    return {reinterpret_cast<__half*>(p), reinterpret_cast<float*>(p ? p + codes : nullptr), codes + ((size_t)rows * 4 + 255) / 256 * 256};
}

template <class T, int VEC>
void rows_launch(const void* x, int64_t ld, int64_t rows, int D, int8_t* out8, __half* out16, int64_t pitch, int ntiles, float* scales, int sms,
                 cudaStream_t st) {
    // two units a thread where there are threads enough, so that one row is quick too
    const int lanes = std::max(8, pow2_at_least((D / VEC + 1) / 2, 256));
    const int64_t blocks = (rows * lanes + 255) / 256;
    k_q8_rows<T, VEC><<<(unsigned)std::min<int64_t>(blocks, 16ll * sms), 256, 0, st>>>(static_cast<const T*>(x), ld, rows, D, lanes, out8, out16, pitch,
                                                                                     ntiles, scales);
}
template <class T>
void rows_launch(const void* x, int64_t ld, int64_t rows, int D, int8_t* out8, __half* out16, int64_t pitch, int ntiles, float* scales, int sms,
                 cudaStream_t st) {
    constexpr int kVec = 16 / (int)sizeof(T);
    if (D % kVec == 0 && aligned(x, 16) && ld % kVec == 0)
        rows_launch<T, kVec>(x, ld, rows, D, out8, out16, pitch, ntiles, scales, sms, st);
    else
        rows_launch<T, 1>(x, ld, rows, D, out8, out16, pitch, ntiles, scales, sms, st);
}

void quantize_rows(const void* x, int64_t ld, int64_t rows, int D, int dtype, int8_t* out8, __half* out16, int64_t pitch, int ntiles, float* scales,
                   int sms, cudaStream_t st) {
    if (dtype == TT_F32)
        rows_launch<float>(x, ld, rows, D, out8, out16, pitch, ntiles, scales, sms, st);
    else if (dtype == TT_BF16)
        rows_launch<__nv_bfloat16>(x, ld, rows, D, out8, out16, pitch, ntiles, scales, sms, st);
    else
        rows_launch<__half>(x, ld, rows, D, out8, out16, pitch, ntiles, scales, sms, st);
}

// [rows][cols] of bytes or f16, rows `pitch` bytes apart, in boxes of 128 bytes x box_rows; outside: 0.
bool make_map2(CUtensorMap* m, const void* p, bool f16, int64_t cols, int64_t rows, int64_t pitch, int box_rows) {
    EncodeTiled enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)pitch};
    const cuuint32_t box[2] = {f16 ? 64u : 128u, (cuuint32_t)box_rows}, one[2] = {1, 1};
    return enc(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(p), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT, bool LONG>
tt_status few_launch(FewArgs8 a, int sms, cudaStream_t st) {
    // warps that share a tile's columns: more of them while the tiles alone would give a warp slot fewer
    // than 4, as long as each keeps four steps
    const int64_t tiles = (a.V + kFewTile - 1) / kFewTile;
    a.ksplit = 1;
    while (a.ksplit < kFewWarps8 && tiles * a.ksplit < 4ll * sms * 2 * kFewWarps8 && a.steps >= 8 * a.ksplit) a.ksplit *= 2;
    const int64_t per = kFewWarps8 / a.ksplit, rounds = (tiles + per - 1) / per;
    return launch_ahead(k_q8_few<NT, LONG>, dim3((unsigned)std::min<int64_t>(rounds, 2 * sms)), kFewThreads, 0, st, a) ? TT_OK : TT_ERR_CUDA;
}

template <int BN>
struct Q8Tag {};

template <int BN>
tt_status scores_launch(Q8Args a, const int8_t* codes, const __half* x, int D, int sms, int dev, cudaStream_t st) {
    CUtensorMap mc, mx;
    if (!make_map2(&mc, codes, false, code_pitch(D), a.V, code_pitch(D), 128) || !make_map2(&mx, x, true, x_pitch(D), a.M, x_pitch(D) * 2, BN))
        return TT_ERR_CUDA;
    a.mtiles = (int)((a.M + BN - 1) / BN);
    a.units = (a.V + 127) / 128 * a.mtiles;
    if (!allow_smem<Q8Tag<BN>>(k_q8_scores<BN>, dev, Q8Shape<BN>::kSmem)) return TT_ERR_CUDA;
    if (Q8Shape<BN>::kShift) {  // the warps that take registers wait for them: they have to be there
        static std::atomic<bool> enough{false};
        cudaFuncAttributes f;
        if (!enough.load(std::memory_order_relaxed)) {
            if (cudaFuncGetAttributes(&f, k_q8_scores<BN>) != cudaSuccess) {
                cudaGetLastError();
                return TT_ERR_CUDA;
            }
            if (f.numRegs < kQ8Regs) return TT_ERR_CUDA;
            enough.store(true, std::memory_order_relaxed);
        }
    }
    return launch_ahead(k_q8_scores<BN>, dim3((unsigned)std::min<int64_t>(a.units, sms * Q8Shape<BN>::kBlocks)), Q8Shape<BN>::kThreads, Q8Shape<BN>::kSmem, st, mc, mx, a) ? TT_OK
                                                                                                                                         : TT_ERR_CUDA;
}

}  // namespace
}  // namespace ttemb

using namespace ttemb;

extern "C" {

int64_t tt_emb_q8_workspace(int64_t rows, int32_t dim) {
    if (q8_sizes(rows, dim, TT_F32) != TT_OK || rows > TT_Q8_MAX_ROWS) return -1;
    return (int64_t)q8_space(rows, dim, nullptr).bytes;
}

tt_status tt_emb_q8_quantize(const void* weight_dev, int64_t weight_stride, int64_t rows, int32_t dim, int32_t dtype, int8_t* codes_dev,
                             float* scales_dev, tt_stream stream) {
    const tt_status s = q8_sizes(rows, dim, dtype);
    if (s != TT_OK) return s;
    if (weight_stride < dim) return TT_ERR_SHAPE;
    if (rows && (!weight_dev || !codes_dev || !scales_dev)) return TT_ERR_ARG;
    if (!aligned(weight_dev, dtype == TT_F32 ? 4 : 2) || !aligned(codes_dev, 16) || !aligned(scales_dev, 4)) return TT_ERR_ARG;
    if (rows == 0) return TT_OK;
    const int sms = head_sms();
    if (sms <= 0) return TT_ERR_CUDA;
    quantize_rows(weight_dev, weight_stride, rows, dim, dtype, codes_dev, nullptr, code_pitch(dim), 0, scales_dev, sms, reinterpret_cast<cudaStream_t>(stream));
    return cudaGetLastError() == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

tt_status tt_emb_q8_scores(const void* x_dev, int64_t x_stride, int64_t rows, int32_t dtype, const int8_t* codes_dev, const float* scales_dev,
                           int64_t vocab, int32_t dim, float* out_dev, int32_t* err_dev, void* ws_dev, size_t ws_bytes, tt_stream stream) {
    const tt_status s = q8_sizes(vocab, dim, dtype);
    if (s != TT_OK) return s;
    if (rows < 0 || rows > TT_Q8_MAX_ROWS || vocab < 1 || x_stride < dim) return TT_ERR_SHAPE;
    if (rows == 0) return TT_OK;
    if (!x_dev || !codes_dev || !scales_dev || !out_dev || !ws_dev) return TT_ERR_ARG;
    if (!aligned(x_dev, dtype == TT_F32 ? 4 : 2) || !aligned(codes_dev, 16) || !aligned(scales_dev, 4) || !aligned(out_dev, 4) || !aligned(err_dev, 4) ||
        !aligned(ws_dev, 256))
        return TT_ERR_ARG;
    const Q8Space w = q8_space(rows, dim, ws_dev);
    if (ws_bytes < w.bytes) return TT_ERR_ARG;
    int dev = 0;
    const int sms = head_sms(&dev);
    if (sms <= 0) return TT_ERR_CUDA;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int nt = few_tiles(rows, dim);
    quantize_rows(x_dev, x_stride, rows, dim, dtype, nullptr, w.x, nt ? few_pitch(dim) : x_pitch(dim), nt, w.xscale, sms, st);
    if (cudaGetLastError() != cudaSuccess) return TT_ERR_CUDA;
    if (nt) {
        FewArgs8 f{};
        f.codes = codes_dev;
        f.pitch = code_pitch(dim);
        f.V = vocab;
        f.scale = scales_dev;
        f.x = reinterpret_cast<const uint4*>(w.x);
        f.xscale = w.xscale;
        f.M = (int)rows;
        f.steps = (int)(few_pitch(dim) / kFewK);
        f.out = out_dev;
        if (nt == 2) return few_launch<2, false>(f, sms, st);
        return dim > 256 ? few_launch<1, true>(f, sms, st) : few_launch<1, false>(f, sms, st);
    }
    Q8Args a{};
    a.M = rows;
    a.V = vocab;
    a.chunks = (dim + kQ8K - 1) / kQ8K;
    a.xscale = w.xscale;
    a.scale = scales_dev;
    a.out = out_dev;
    a.wait_ns = head_wait_limit();
    a.err = err_dev;
    // The narrowest tile that holds the rows, 192 beyond.  By 60000 x 4096, us: 32 rows 52 (the next wider tile 54), 64 rows 59 (narrower 81,
    // wider 76), 65 rows 71 (84, 92), 128 rows 78 (91, 95), 192 rows 98 (125), 384 rows 158 (174 in tiles of 128), 512 rows 206 (226).
    // 193 to 256 rows would be quicker in two tiles of 128 (256 rows 125, 149 this way).
    if (rows <= 32) return scores_launch<32>(a, codes_dev, w.x, dim, sms, dev, st);
    if (rows <= 64) return scores_launch<64>(a, codes_dev, w.x, dim, sms, dev, st);
    if (rows <= 128) return scores_launch<128>(a, codes_dev, w.x, dim, sms, dev, st);
    return scores_launch<192>(a, codes_dev, w.x, dim, sms, dev, st);
}

}  // extern "C"
