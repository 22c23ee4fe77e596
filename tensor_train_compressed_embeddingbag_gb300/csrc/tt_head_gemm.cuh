// tt_head_gemm.cuh -- the vocabulary head's products of large matrices: scores with a
// softmax epilogue, dz of a piece of the vocabulary, and the two gradient products.
#pragma once

#include "tt_head.cuh"

namespace ttemb {

constexpr int kEpiWarps = 16;
constexpr int kGemmThreads = (4 + kEpiWarps) * 32;  // warp 0: TMA, 1: MMA, 2: tensor memory, 4..: epilogue
constexpr int kParts = kEpiWarps / 4;               // column parts of a tile, a warp per part and 32 rows
constexpr int kBK = 64;            // K depth of a stage: one 128-byte swizzled row

enum Epi { kEpiStats = 0, kEpiDz = 1, kEpiOut = 2, kEpiStatsLong = 3 };  // the last: 16-bit types, more than kLongChunks of K
constexpr int kLongChunks = 8;  // 512 of K; 1,024 takes the same time and has twice the error

struct GemmArgs {
    int64_t M, N;      // valid rows and columns of the product
    int mtiles, ntiles;
    int strip;         // column tiles per unit (kEpiStats), else 1
    int nstrips;
    int splits;        // K ranges (kEpiOut), else 1
    int chunks;        // K chunks of 64
    int64_t units;
    int fmt;           // 16-bit type of the operands: 0 f16, 1 bf16
    uint64_t wait_ns;
    int* err;
    // scales: exponents of the operands' power-of-two scales come from these bits
    const uint32_t* amax_a;
    const uint32_t* amax_b;
    const int* row_exp;  // exponents of A's rows (with amax_a's), else null
    // SPLIT: exponents of the table's 128 x 128 blocks, kb to a row of blocks: scores: B's
    // rows by K; dhidden: K by columns; dweight: null
    const int* wexp;
    int kb;
    float ctemp;         // log2(e) / T
    // kEpiStats
    float2* part;        // [M][nstrips][kParts] (maximum in log2 units, sum)
    // kEpiDz
    const float* nlse;   // per row -lse in log2 units, and its scale (kEpiOut: null, or 0 for rows that are 0)
    const float* scale;
    uint16_t* dz;        // [pieces][M][dz_pitch]
    int64_t dz_pitch, dz_piece;
    // kEpiOut
    OutArgs to;
};

template <int BN, bool SPLIT>
struct GemmShape {
    static constexpr int PC = SPLIT ? 2 : 1;
    static constexpr uint32_t kA = 128 * 128, kB = BN * 128;  // a chunk of one piece
    static constexpr uint32_t kStage = PC * (kA + kB);        // A hi, A lo, B hi, B lo
    static constexpr int kStages = 192 * 1024 / kStage;
    static constexpr uint32_t kRing = kStages * kStage;       // then 2 KB per epilogue warp (put_rows)
    static constexpr size_t kSmem = (size_t)kRing + kEpiWarps * 2048 + 1024;
    static constexpr int kAcc = PC * BN;                      // tensor-memory columns of an accumulator
    static_assert(kSmem + 512 <= 227 * 1024 && 2 * kAcc <= 512, "shared and tensor memory");
};

// C[m, n] = sum_k A[m, k] B[n, k] by 128 x BN tiles, a persistent block per SM: one
// thread feeds a ring of stages by TMA, one issues the MMAs into one of two
// accumulators in tensor memory, sixteen warps read the other out, a quarter of its
// columns and 32 of its rows each, a row per lane.
//
// SPLIT (fp32 operands in two pieces).  The pieces of B lie one behind the other, so
// A hi [B hi | B lo] is one MMA of twice the columns; A lo B hi adds to its second half,
// which holds the small products.
//
// Ranges.  The tensor core's fp32 accumulation cuts off the bits below its accumulator
// instead of rounding them, so the error of a long sum grows with its length and always in
// one direction.  Where the result is fp32 (fp32 operands; scores of 16-bit ones, whose lse
// is) an accumulator therefore holds kRange K chunks only, and the epilogue adds the ranges up in
// registers, rounding to nearest.  For 16-bit scores that is no slower, as the epilogue lets an
// accumulator go before its exponentials: bf16 4096 x 131072 x 2048 1186 us (1217 in one range),
// 300 x 20000 x 4096 83 (88); the error of lse falls from 5.8e-7 to 1.4e-7 and from 1.3e-6 to
// 1.5e-7.  dz and the gradients of 16-bit types are rounded to 16 bits, far above that.
//
// Bound by the tensor cores from some hundred rows and columns on (their pipe 79% busy in
// the scores of 2048 x 16384 x 2048 bf16, 71 in dz, 75 in dhidden, 64 in dweight).  Measured
// within whole steps, bf16 4096 x 131072 x 2048, 2.2 TFLOP a product: scores 1215 us (1810
// TFLOP/s), dz 1367 (1610), dhidden 1446 (1520), dweight 1486 (1480); f16 2047 x 50001 x 1024
// scores 126 us (1660); fp32 283 x 37955 x 1451 scores 91 us (340, three products each).  With few
// hidden rows it is a stream: bf16 8 x 200000 x 1024 reads the table for dhidden at 5.4 TB/s
// (76 us) and writes dweight at 5.3 (78 us).
template <int BN, bool AMN, bool BMN, int EPI, bool SPLIT>
__global__ void __launch_bounds__(kGemmThreads, 1)
    k_head_gemm(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
                const __grid_constant__ GemmArgs a) {
    using S = GemmShape<BN, SPLIT>;
    static_assert(BN % (32 * kParts) == 0 && (!SPLIT || BN <= 128), "the ranges' sums stay in registers");
    constexpr bool STATS = EPI == kEpiStats || EPI == kEpiStatsLong;
    constexpr bool RANGES = SPLIT || EPI == kEpiStatsLong;
    constexpr int kRange = SPLIT ? 2 : kLongChunks;  // SPLIT: 128 of K
    constexpr int kCh = BN / kParts / 32;  // 32-column chunks of a part
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t full[S::kStages], empty[S::kStages], accfull[2], accempty[2], drain;
    __shared__ uint32_t tmem_slot;
    __shared__ int gave_up_s;
    volatile int* gave_up = &gave_up_s;
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const bool lead = lane == 0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&accfull[i], 1);
            mbar_init(&accempty[i], kEpiWarps);
        }
        mbar_init(&drain, 1);
        gave_up_s = 0;
    }
    if (warp == 2) tc_alloc(&tmem_slot, 2 * S::kAcc);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    uint32_t it = 0;   // stages fed (TMA thread) or consumed (MMA thread)
    uint32_t acc = 0;  // accumulators filled (MMA thread) or read (epilogue)
    bool ok = true;

    // unit -> row tile, column tiles, K range, and which split or strip it is
    auto unit = [&](int64_t u, int& m, int& n0, int& n1, int& kb, int& ke, int& split) {
        if (EPI == kEpiOut) {  // column tiles fastest: blocks that run together share rows of A
            const int64_t tiles = (int64_t)a.mtiles * a.ntiles;
            split = (int)(u / tiles);
            const int64_t t = u - split * tiles;
            m = (int)(t / a.ntiles);
            n0 = (int)(t - (int64_t)m * a.ntiles);
            n1 = n0 + 1;
            kb = (int)((int64_t)a.chunks * split / a.splits);
            ke = (int)((int64_t)a.chunks * (split + 1) / a.splits);
        } else {  // row tiles fastest: blocks that run together share rows of the table
            const int s = (int)(u / a.mtiles);
            m = (int)(u - (int64_t)s * a.mtiles);
            n0 = s * a.strip;
            n1 = min(n0 + a.strip, a.ntiles);
            kb = 0;
            ke = a.chunks;
            split = s;
        }
    };

    if (warp == 0) {
        for (int64_t u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
            int m, n0, n1, kb, ke, split;
            unit(u, m, n0, n1, kb, ke, split);
            for (int n = n0; ok && n < n1; ++n)
                for (int kc = kb; kc < ke; ++kc, ++it) {
                    const uint32_t st = it % S::kStages;
                    ok = head_wait(&empty[st], ((it / S::kStages) & 1) ^ 1, a.wait_ns, gave_up);
                    if (!ok) break;
                    if (lead) {
                        const uint32_t sa = base + st * S::kStage, sb = sa + S::PC * S::kA;
                        bulk_expect(&full[st], S::kStage);
#pragma unroll
                        for (int z = 0; z < S::PC; ++z) {
                            if (AMN) {
                                tma_load3(sa + z * S::kA, &mapA, m * 128, kc * kBK, z, &full[st]);
                                tma_load3(sa + z * S::kA + 8192, &mapA, m * 128 + 64, kc * kBK, z, &full[st]);
                            } else {
                                tma_load3(sa + z * S::kA, &mapA, kc * kBK, m * 128, z, &full[st]);
                            }
                            if (BMN) {
#pragma unroll
                                for (int j = 0; j < BN / 64; ++j)
                                    tma_load3(sb + z * S::kB + j * 8192, &mapB, n * BN + j * 64, kc * kBK, z, &full[st]);
                            } else {
                                tma_load3(sb + z * S::kB, &mapB, kc * kBK, n * BN, z, &full[st]);
                            }
                        }
                    }
                    __syncwarp();
                }
        }
    } else if (warp == 1) {
        const uint32_t idesc = idesc_f16(128, BN, a.fmt, AMN, BMN), idesc2 = idesc_f16(128, S::PC * BN, a.fmt, AMN, BMN);
        const uint32_t da0 = desc_lo(base, AMN ? 8192 : kNoLbo), db0 = desc_lo(base + S::PC * S::kA, BMN ? 8192 : kNoLbo);
        for (int64_t u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
            int m, n0, n1, kb, ke, split;
            unit(u, m, n0, n1, kb, ke, split);
            for (int n = n0; ok && n < n1; ++n)
                for (int r0 = kb; ok && r0 < ke; r0 = RANGES ? (r0 / kRange + 1) * kRange : ke, ++acc) {
                    const int steps = RANGES ? min((r0 / kRange + 1) * kRange, ke) - r0 : ke - kb;
                    const uint32_t buf = acc & 1, d = tmem + buf * S::kAcc;
                    ok = head_wait(&accempty[buf], ((acc >> 1) & 1) ^ 1, a.wait_ns, gave_up);
                    if (!ok) break;
                    tc_fence_after();
                    for (int c = 0; c < steps; ++c, ++it) {
                        const uint32_t st = it % S::kStages;
                        ok = head_wait(&full[st], (it / S::kStages) & 1, a.wait_ns, gave_up);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t da = da0 + st * (S::kStage >> 4), db = db0 + st * (S::kStage >> 4);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t ak = da + k * ((AMN ? 2048 : 32) >> 4), bk = db + k * ((BMN ? 2048 : 32) >> 4);
                            mma_f16(d, ak, bk, idesc2, c > 0 || k > 0, lead);
                            if (SPLIT) mma_f16(d + BN, ak + (S::kA >> 4), bk, idesc, true, lead);
                        }
                        mma_commit(&empty[st], lead);
                    }
                    if (ok) mma_commit(&accfull[buf], lead);
                }
        }
    } else if (warp >= 4) {
        const int part = (warp - 4) >> 2, quad = warp & 3;
        const int r = quad * 32 + lane;
        uint4* const buf = reinterpret_cast<uint4*>(raw + (base - smem_addr(raw)) + S::kRing + (warp - 4) * 2048);
        const int e = amax_exp(a.amax_a) + amax_exp(a.amax_b);
        const float c = a.ctemp;
        for (int64_t u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
            int m, n0, n1, kb, ke, split;
            unit(u, m, n0, n1, kb, ke, split);
            const int64_t row = (int64_t)m * 128 + r;
            const bool in = row < a.M;
            float run_m = -INFINITY, run_s = 0.f;
            int er = e;  // the scales that the row's sums are freed of
            float2 rc = make_float2(0.f, 0.f);
            if ((SPLIT || EPI == kEpiOut) && a.row_exp && in) er += a.row_exp[row];
            const Pow2 sc(SPLIT ? 0 : -er);
            if (EPI == kEpiDz && in) rc = make_float2(a.nlse[row], a.scale[row]);
            const bool zero = EPI == kEpiOut && a.scale && in && a.scale[row] == 0.f;
            for (int n = n0; ok && n < n1; ++n) {
                const int64_t col0 = (int64_t)n * BN + part * (BN / kParts);
                // 32 finished columns of this thread's row, the first of them `col`
                auto finish = [&](float (&v)[32], int64_t col) {
                    if (STATS) {
                        take_scores(v, a.N - col, c, run_m, run_s);
                    } else if (EPI == kEpiDz) {
                        if (col < a.dz_pitch && row - lane < a.M) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] = rc.y == 0.f ? 0.f : rc.y * ex2(fmaf(v[j], c, rc.x));
                            uint16_t* to = a.dz + (row - lane) * a.dz_pitch + col;
                            put_rows_16(buf, v, reinterpret_cast<uint8_t*>(to), a.dz_pitch * 2, a.M - (row - lane), SPLIT ? 0 : a.fmt);
                            if (SPLIT) {
#pragma unroll
                                for (int j = 0; j < 32; ++j) v[j] -= __half2float(__float2half_rn(v[j]));
                                put_rows_16(buf, v, reinterpret_cast<uint8_t*>(to + a.dz_piece), a.dz_pitch * 2, a.M - (row - lane), 0);
                            }
                        }
                    } else if (col < a.N && row - lane < a.M) {
                        if (zero) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] = 0.f;
                        }
                        store_out(a.to, buf, split, row - lane, col, a.M, a.N, v, sc);
                    }
                };
                if (SPLIT) {
                    float sum[kCh][32];
                    for (int r0 = kb; ok && r0 < ke; r0 = (r0 / kRange + 1) * kRange, ++acc) {
                        const uint32_t buf = acc & 1;
                        ok = head_wait(&accfull[buf], (acc >> 1) & 1, a.wait_ns, gave_up);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t t0 = tmem + buf * S::kAcc + ((uint32_t)(quad * 32) << 16) + part * (BN / kParts);
                        const int we = a.wexp ? __ldg(&a.wexp[EPI == kEpiOut ? (int64_t)(r0 / kRange) * a.kb + n : (int64_t)n * a.kb + r0 / kRange]) : 0;
                        const Pow2 f(-er - we);
#pragma unroll
                        for (int ch = 0; ch < kCh; ++ch) {
                            float v[32], small[16];
                            tm_ld32(t0 + ch * 32, v);
                            tm_wait_ld(v);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                tm_read16(t0 + BN + ch * 32 + h * 16, small);
#pragma unroll
                                for (int j = 0; j < 16; ++j) v[h * 16 + j] += small[j];
                            }
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] *= f.b;
#pragma unroll
                            for (int j = 0; j < 32; ++j) sum[ch][j] = r0 == kb ? v[j] * f.a : fmaf(v[j], f.a, sum[ch][j]);
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&accempty[buf]);
                    }
                    if (!ok) break;
#pragma unroll
                    for (int ch = 0; ch < kCh; ++ch) finish(sum[ch], col0 + ch * 32);
                } else if (RANGES) {
                    float sum[kCh][32];
#pragma unroll
                    for (int ch = 0; ch < kCh; ++ch)
#pragma unroll
                        for (int j = 0; j < 32; ++j) sum[ch][j] = 0.f;
#pragma unroll 1
                    for (int r0 = kb; ok && r0 < ke; r0 += kRange, ++acc) {
                        const uint32_t buf = acc & 1;
                        ok = head_wait(&accfull[buf], (acc >> 1) & 1, a.wait_ns, gave_up);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t t0 = tmem + buf * S::kAcc + ((uint32_t)(quad * 32) << 16) + part * (BN / kParts);
#pragma unroll
                        for (int h = 0; h < 4 * kCh; ++h) {
                            float v[8];
                            tm_read8(t0 + h * 8, v);
#pragma unroll
                            for (int j = 0; j < 8; j += 2) add2(sum[h / 4][(h & 3) * 8 + j], sum[h / 4][(h & 3) * 8 + j + 1], v[j], v[j + 1]);
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&accempty[buf]);
                    }
                    if (!ok) break;
#pragma unroll
                    for (int ch = 0; ch < kCh; ++ch) finish(sum[ch], col0 + ch * 32);
                } else {
                    const uint32_t buf = acc & 1;
                    ok = head_wait(&accfull[buf], (acc >> 1) & 1, a.wait_ns, gave_up);
                    if (!ok) break;
                    ++acc;
                    tc_fence_after();
                    const uint32_t t0 = tmem + buf * S::kAcc + ((uint32_t)(quad * 32) << 16) + part * (BN / kParts);
                    // the next 32 columns are on their way while these are worked on; not for
                    // gradients, whose stores want the registers (bf16 dweight of 8 x 200000 x
                    // 1024: 78 us, 105 with it)
                    constexpr int kAhead = EPI != kEpiOut;
                    float v[1 + kAhead][32];
                    if (kAhead) {
                        tm_ld32(t0, v[0]);
                        tm_wait_ld(v[0]);
                    }
#pragma unroll
                    for (int ch = 0; ch < kCh; ++ch) {
                        if (kAhead && ch + 1 < kCh) tm_ld32(t0 + (ch + 1) * 32, v[(ch + 1) & kAhead]);
                        if (!kAhead) {
                            tm_ld32(t0 + ch * 32, v[0]);
                            tm_wait_ld(v[0]);
                        }
                        finish(v[ch & kAhead], col0 + ch * 32);
                        if (kAhead && ch + 1 < kCh) tm_wait_ld(v[(ch + 1) & kAhead]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&accempty[buf]);
                }
            }
            if (STATS && ok && in)
                a.part[(row * a.nstrips + split) * kParts + part] = make_float2(run_m, run_s);
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
            for (uint32_t i = it > S::kStages ? it - S::kStages : 0; i < it; ++i)
                head_drain(&full[i % S::kStages], (i / S::kStages) & 1);
        if (threadIdx.x == 32) {
            mma_commit(&drain, true);
            head_drain(&drain, 0);
        }
        __syncwarp();
        __syncthreads();
    }
    tc_fence_after();
    if (warp == 2) tc_dealloc(tmem, 2 * S::kAcc);
}

}  // namespace ttemb
