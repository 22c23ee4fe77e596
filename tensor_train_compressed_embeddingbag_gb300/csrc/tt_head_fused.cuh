// tt_head_fused.cuh -- the vocabulary head for widths up to 128: scores, and dz, never
// leave the chip.
//
//   kLse      max and sum of exp of z[n, v]        resident rows: hidden, streamed: weight
//   kDhidden  sum_v dz[n, v] weight[v]             resident rows: hidden, streamed: weight
//   kDweight  sum_n dz[n, v] hidden[n]             resident rows: weight, streamed: hidden
//
// One kernel for the three: a block holds 128 resident rows X and streams tiles of BY rows
// Y.  Per tile, S = X Y^T (tensor cores, K = D), warps turn S into dz (one exponential an
// element) and write it back to tensor memory in 16 bits, where it is the A operand of
// OUT += dz Y (K = BY); the same bytes of Y in shared memory are read K-major by the
// first product and MN-major by the second.  At these widths dz in memory would cost
// more than forming S twice: 6 bytes of traffic an element (written once, read twice)
// against 2 D FLOP and one exponential.
//
// A tile's way through S, dz and OUT is long: every hand-over between the tensor cores
// and the warps costs one to four hundred cycles, and so does what an issuing warp does
// around a tile's MMAs (its waits and commits).  So two warps issue S, taking tiles in
// turn, and one issues OUT; S has three buffers, two sets of dz warps take tiles in turn,
// and what a dz warp needs of memory (lse and scale of the hidden rows, its block's first
// targets) is fetched while it works on the tile before.  X (but for fp32 at D > 64, where shared
// memory is full) and OUT (where tensor memory has room) have two buffers, and eight
// further warps take OUT to memory, so segments follow each other without a gap.
//
// SPLIT (fp32: every operand as f16 hi + lo): three products each; OUT covers two tiles of
// Y at a time, its small products in columns of their own where there is room, and its
// sums are kept in the storing warps' registers (k_head_gemm says why).  Sums read
// every tile instead of every second one: dweight of 512 x 1,000,000 x 64 took 315 us,
// here 256.
//
// Measured, us and TFLOP/s of its 2 N V D (kLse) or 4 N V D products (SPLIT: x 3):
// bf16 4096 x 100003 x 128 dhidden 119 (1760), dweight 142 (1480); fp32 512 x 1,000,000 x
// 64 lse 148 (1330), dhidden 241 (1630), dweight 261 (1510).  The tensor pipe is 60 to 70%
// busy and what bounds them; the rest is fill and drain of the tiles' way above.
#pragma once

#include "tt_head.cuh"
#include "tt_head_pipe.cuh"

namespace ttemb {

// The elements of dz that have a target, by 32 x 32 block of (hidden row, table row): a
// block holds two of them, how many there are, and the rest in a list.  Where many rows of
// a batch share popular items the list is long and every step of it a memory latency:
// then the 32 rows' entries are gone through instead, a row per lane, four loads at a
// time (a bf16 batch of 4096 over 25,003 items drawn by popularity, D = 128: dweight 59 us,
// with lists alone 64; uniform ones change nothing).  An element's place in its block is (n & 31) | (v & 31) << 5; its value
// is under the batch's scale.  All zero: none.
struct __align__(16) TargetBlock {
    uint32_t meta;  // places of the two (bits 0..9 and 10..19), bits 20..31: how many elements
    float val[2];
    int next;       // 1 + index of the list's first entry, 0: none
};
struct __align__(16) TargetEntry {
    int at;
    float val;
    int next;
    int pad;
};

// Called once per element.
__device__ __forceinline__ void add_target(TargetBlock* b, TargetEntry* ents, int e, int at, float val) {
    const uint32_t k = atomicAdd(&b->meta, 1u << 20) >> 20;
    if (k < 2) {
        atomicOr(&b->meta, (uint32_t)at << (10 * k));
        b->val[k] = val;
    } else {
        TargetEntry x;
        x.at = at;
        x.val = val;
        x.pad = 0;
        x.next = atomicExch(&b->next, e + 1);
        ents[e] = x;
    }
}

struct FusedArgs {
    int64_t X, Y;   // resident and streamed rows
    int D;
    Runs runs;
    int fmt;
    uint64_t wait_ns;
    int* err;
    const uint32_t* amax_h;  // power-of-two scales of hidden and dz (null: none)
    const uint32_t* amax_z;
    const int* row_exp;      // SPLIT, kLse: hidden's, per row instead
    const int* wexp;         // SPLIT: weight's, per two streamed tiles (D <= 64: 256 rows, else 128)
    float ctemp;             // log2(e) / T
    float2* part;            // kLse: [X][slots][kParts] (maximum in log2 units, sum), a slot per run
    int slots;
    const float* nlse;       // per hidden row -lse in log2 units, and its scaled weight (kDhidden: by the
    const float* scale;      //   row's own power of two, kDweight: by the batch's); up to a multiple of 128 rows
    const int* zexp;         // kDhidden: exponent of the row's own scale over the batch's (null: 0),
    const float* to_own;     //   and what takes an element of dz from the batch's scale to it, as scale has it
    const TargetBlock* blocks;  // [vblocks][nblocks]
    const TargetEntry* ents;
    const int* ids;             // [K][hidden rows] the rows' entries (-1: none) and their elements of dz under the batch's scale
    const float* dzt;
    int K;
    int64_t rows;
    Residue low;             // kDhidden: for k_head_join
    int nblocks, vblocks;
    OutArgs to;              // whole segments; others, and all with `low`, as fp32 sums to
    float* partial;          //   [blocks][2][128][to.pp]: the run's first segment, its last
};

enum FusedMode { kLse = 0, kDhidden = 1, kDweight = 2 };

template <int DT, bool SPLIT>
struct FusedShape {
    static constexpr int BY = SPLIT && DT == 128 ? 64 : 128;
    static constexpr int PC = SPLIT ? 2 : 1, DB = DT / 64;
    static constexpr int XB = SPLIT && DT == 128 ? 1 : 2;
    static constexpr int kStages = DT == 64 && !SPLIT ? 6 : 4;
    static constexpr uint32_t kXBlock = 128 * 128, kYBlock = BY * 128;  // 64 columns of a tile
    static constexpr uint32_t kX = PC * DB * kXBlock, kY = PC * DB * kYBlock;
    static constexpr size_t kSmem = (size_t)XB * kX + (size_t)kStages * kY + 1024;
    // warp 0: TMA, 1 and 2: S, 3: OUT product, 4..11: OUT to memory, 12..: dz
    static constexpr int kDzSet = BY / 16, kDzWarps = 2 * kDzSet, kThreads = (12 + kDzWarps) * 32;
    static constexpr int kParts = 2 * (BY / 64);  // kLse: pairs per row and unit, one of each dz warp of the row
    // tensor memory: three S, then OUT (fp32 at D <= 64: hi hi and the two small products
    // in columns of their own)
    static constexpr int NS = 3, kOut = SPLIT && DT == 64 ? 128 : DT, OB = (512 - NS * BY) / kOut >= 2 ? 2 : 1;
    static constexpr uint32_t kOutCol = NS * BY;
    static_assert(NS * BY + OB * kOut <= 512, "tensor memory");
};

// The target elements of a 32 x 32 block of dz, after its warp has written the block to
// tensor memory from t0 on: each replaces one 16-bit half (SPLIT: and its lo part, 16
// columns further) of one column.  nb, vb: which block; COLS: hidden rows are columns; else
// to_own: from the batch's scale to that of this lane's row.
template <bool SPLIT, bool COLS>
__device__ __noinline__ void put_targets(const FusedArgs& a, uint32_t t0, uint4 b, int nb, int vb, float to_own) {
    const int lane = threadIdx.x & 31, count = (int)(b.x >> 20);
    auto put = [&](int col, bool mine, float val) {
        if (!COLS) val *= to_own;
        const uint32_t hi = pack16(val, 0.f, SPLIT ? 0 : a.fmt) & 0xFFFFu, sh = (uint32_t)(col & 1) * 16;
        uint32_t w = tm_read1(t0 + (col >> 1));
        if (mine) w = (w & ~(0xFFFFu << sh)) | hi << sh;
        tm_write1(t0 + (col >> 1), w);
        if (SPLIT) {
            const uint32_t lo = pack16(val - unpack_f16(hi).x, 0.f, 0) & 0xFFFFu;
            w = tm_read1(t0 + 16 + (col >> 1));
            if (mine) w = (w & ~(0xFFFFu << sh)) | lo << sh;
            tm_write1(t0 + 16 + (col >> 1), w);
        }
        tm_wait_st();  // the next may be in the same column
    };
    auto place = [&](int at, float val) {
        const int n = at & 31, v = at >> 5;
        put(COLS ? n : v, lane == (COLS ? v : n), val);
    };
    if (a.K >= 2 * (count - 2)) {  // count - 2 steps of the list, or K / 4 rounds of loads
        place(b.x & 1023, __uint_as_float(b.y));
        if (count > 1) place((b.x >> 10) & 1023, __uint_as_float(b.z));
#pragma unroll 1
        for (int e = (int)b.w; e;) {
            const int4 t = __ldg(reinterpret_cast<const int4*>(a.ents + (e - 1)));
            place(t.x, __int_as_float(t.y));
            e = t.z;
        }
        return;
    }
    const int64_t n = (int64_t)nb * 32 + lane;
#pragma unroll 1
    for (int k0 = 0; k0 < a.K; k0 += 4) {
        int off[4];
        float val[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = n < a.rows && k0 + i < a.K;
            off[i] = in ? __ldg(&a.ids[(k0 + i) * a.rows + n]) - vb * 32 : -1;
            val[i] = in ? __ldg(&a.dzt[(k0 + i) * a.rows + n]) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t m = __ballot_sync(0xffffffffu, (uint32_t)off[i] < 32u);
            while (m) {
                const int from = __ffs(m) - 1, o = __shfl_sync(0xffffffffu, off[i], from);
                if (COLS) {
                    const float x = __shfl_sync(0xffffffffu, val[i], from);
                    put(from, lane == o, x);
                    m &= m - 1;
                } else {  // all rows with that column at once
                    put(o, off[i] == o, val[i]);
                    m &= ~__ballot_sync(0xffffffffu, off[i] == o);
                }
            }
        }
    }
}

// kLse has no OUT: a tile's dz warps free its S, and its stage is free once S is formed (tt_head_pipe.cuh).
template <int DT, bool SPLIT, int MODE>
__global__ void __launch_bounds__((FusedShape<DT, SPLIT>::kThreads), 1)
    k_head_fused(const __grid_constant__ CUtensorMap mapX, const __grid_constant__ CUtensorMap mapY,
                 const __grid_constant__ FusedArgs a) {
    using S = FusedShape<DT, SPLIT>;
    using Pipe = TilePipe<S::kStages, S::NS, MODE == kLse>;
    constexpr bool COLS = MODE == kDweight;  // hidden rows are columns of S: lse and scale go by column
    constexpr int BY = S::BY, NS = S::NS, OB = S::OB, kSegs = SPLIT ? 3 : 1;
    extern __shared__ uint8_t raw[];
    // of the tiles, as Pipe has them: loaded, formed, done, turned
    __shared__ uint64_t xfull[S::XB], xempty[S::XB], yfull[S::kStages], sfull[Pipe::kFormed], odone[S::kStages];
    __shared__ uint64_t pready[Pipe::kTurned], ofull[OB], oempty[OB], drain[3];
    // what a dz warp needs of memory for a tile, and for the next: -lse and scale of its
    // columns (COLS) or rows (and to_own), the targets of its two 32 x 32 blocks
    struct Ahead {
        float nlse[COLS ? 64 : 32], scale[64];  // not COLS: 32 scales, then 32 of to_own
        uint4 blk[2];
        int wexp[4];  // the first: scale of the tile's table rows
    };
    __shared__ __align__(16) Ahead ahead[S::kDzWarps][2];
    __shared__ uint4 rows_out[MODE == kLse ? 1 : 8][128];  // put_rows of the warps that store OUT
    static_assert(S::kSmem + sizeof(ahead) + sizeof(rows_out) + 512 <= 227 * 1024, "shared memory");
    __shared__ uint32_t tmem_slot;
    __shared__ int gave_up_s;
    volatile int* gave_up = &gave_up_s;
    const auto formed = [&](uint32_t t) { return head_wait(&sfull[Pipe::formed(t).bar], Pipe::formed(t).n & 1, a.wait_ns, gave_up); };
    const auto done = [&](uint32_t t) { return head_wait(&odone[Pipe::done(t).bar], Pipe::done(t).n & 1, a.wait_ns, gave_up); };
    const auto turned = [&](uint32_t t) { return head_wait(&pready[Pipe::turned(t).bar], Pipe::turned(t).n & 1, a.wait_ns, gave_up); };
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    const uint32_t ybase = base + S::XB * S::kX;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const bool lead = lane == 0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::XB; ++i) {
            mbar_init(&xfull[i], 1);
            mbar_init(&xempty[i], 2);
        }
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&yfull[i], 1);
            mbar_init(&odone[i], 1);
        }
        for (int i = 0; i < Pipe::kFormed; ++i) mbar_init(&sfull[i], 1);
        for (int i = 0; i < Pipe::kTurned; ++i) mbar_init(&pready[i], S::kDzSet);
        for (int i = 0; i < OB; ++i) {
            mbar_init(&ofull[i], 1);
            mbar_init(&oempty[i], 8);
        }
        for (int i = 0; i < 3; ++i) mbar_init(&drain[i], 1);
        gave_up_s = 0;
    }
    if (warp == 2) tc_alloc(&tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    // The tiles of this block, in order; y0 .. y1 is the segment that tile (x, y) is in.
    struct Walk {
        int left, x, y, y0, y1;  // left: tiles to go, this one counted; 0: none
    };
    auto seg_end = [&](Walk& w) { w.y1 = min(a.runs.ytiles, w.y0 + w.left); };
    auto step = [&](Walk& w) {
        --w.left;
        if (++w.y == w.y1) {
            ++w.x;
            w.y0 = w.y = 0;
            seg_end(w);
        }
    };
    Walk w;
    {
        const int64_t t0 = a.runs.begin(blockIdx.x);
        w.left = (int)(a.runs.begin(blockIdx.x + 1) - t0);
        w.x = (int)(t0 / a.runs.ytiles);
        w.y0 = w.y = (int)(t0 - (int64_t)w.x * a.runs.ytiles);
        seg_end(w);
    }
    bool ok = true;
    uint32_t g = 0, xu = 0;  // tiles and segments fed (TMA warp) or taken (the others)

    if (warp == 0) {
        for (; w.left; step(w), ++g) {
            if (w.y == w.y0) {
                const uint32_t b = xu % S::XB;
                ok = head_wait(&xempty[b], ((xu / S::XB) & 1) ^ 1, a.wait_ns, gave_up);
                if (!ok) break;
                if (lead) {
                    bulk_expect(&xfull[b], S::kX);
                    for (int i = 0; i < S::PC * S::DB; ++i)
                        tma_load3(base + b * S::kX + i * S::kXBlock, &mapX, (i % S::DB) * 64, w.x * 128, i / S::DB, &xfull[b]);
                }
                __syncwarp();
                ++xu;
            }
            const uint32_t st = g % S::kStages;
            ok = g < S::kStages || done(g - S::kStages);
            if (!ok) break;
            if (lead) {
                bulk_expect(&yfull[st], S::kY);
                for (int i = 0; i < S::PC * S::DB; ++i)
                    tma_load3(ybase + st * S::kY + i * S::kYBlock, &mapY, (i % S::DB) * 64, w.y * BY, i / S::DB, &yfull[st]);
            }
            __syncwarp();
        }
    } else if (warp == 1 || warp == 2) {
        const uint32_t idesc = idesc_f16(128, BY, a.fmt, false, false), turn = warp - 1;
        const int ksteps = (a.D + 15) / 16;
        for (; w.left; ++g) {
            const uint32_t b = xu % S::XB, st = g % S::kStages, sb = g % NS;
            if (w.y == w.y0) {
                ok = head_wait(&xfull[b], (xu / S::XB) & 1, a.wait_ns, gave_up);
                if (!ok) break;
            }
            if ((g & 1) == turn) {
                if (g >= NS) ok = MODE == kLse ? turned(g - NS) : done(g - NS);  // S of tile g - NS is done with
                ok = ok && head_wait(&yfull[st], (g / S::kStages) & 1, a.wait_ns, gave_up);
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = tmem + sb * BY;
#pragma unroll
                for (int seg = 0; seg < kSegs; ++seg) {
                    const uint32_t sx = desc_lo(base + b * S::kX + (SPLIT && seg == 0 ? S::DB * S::kXBlock : 0), kNoLbo);
                    const uint32_t sy = desc_lo(ybase + st * S::kY + (SPLIT && seg == 1 ? S::DB * S::kYBlock : 0), kNoLbo);
#pragma unroll
                    for (int k = 0; k < DT / 16; ++k)
                        if (k < ksteps)
                            mma_f16(d, sx + (((k >> 2) * S::kXBlock + (k & 3) * 32) >> 4),
                                    sy + (((k >> 2) * S::kYBlock + (k & 3) * 32) >> 4), idesc, seg > 0 || k > 0, lead);
                }
                mma_commit(&sfull[Pipe::formed(g).bar], lead);
                if (MODE == kLse) mma_commit(&odone[st], lead);
            }
            if (w.y + 1 == w.y1) {
                mma_commit(&xempty[b], lead);  // nothing but S reads X
                ++xu;
            }
            step(w);
        }
    } else if (MODE != kLse && warp == 3) {
        const uint32_t idesc = idesc_f16(128, DT, a.fmt, false, true), idesc2 = idesc_f16(128, 2 * DT, a.fmt, false, true);
        uint32_t fl = 0;
        for (; w.left; step(w), ++g) {
            const uint32_t st = g % S::kStages, sb = g % NS, ob = fl % OB;
            const bool first = w.y == w.y0 || (SPLIT && !(w.y & 1)), last = w.y + 1 == w.y1 || (SPLIT && (w.y & 1));
            if (first) ok = head_wait(&oempty[ob], ((fl / OB) & 1) ^ 1, a.wait_ns, gave_up);
            ok = ok && turned(g);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem + S::kOutCol + ob * S::kOut, p = tmem + sb * BY;
            const uint32_t sy = desc_lo(ybase + st * S::kY, S::kYBlock);
#pragma unroll
            for (int k = 0; k < BY / 16; ++k) {
                const uint32_t pa = p + (k >> 1) * 32 + (k & 1) * 8, yb = sy + (k * 2048 >> 4);
                if (SPLIT && DT == 64) {
                    // the two pieces of Y lie one behind the other: hi [hi | lo] is one MMA of
                    // twice the columns, and the second half takes lo hi as well
                    mma_f16_ta(d, pa, yb, idesc2, !first || k > 0, lead);
                    mma_f16_ta(d + DT, pa + 16, yb, idesc, true, lead);
                } else if (SPLIT) {
                    const uint32_t yl = yb + (S::DB * S::kYBlock >> 4);
                    mma_f16_ta(d, pa + 16, yb, idesc, !first || k > 0, lead);
                    mma_f16_ta(d, pa, yl, idesc, true, lead);
                    mma_f16_ta(d, pa, yb, idesc, true, lead);
                } else {
                    mma_f16_ta(d, pa, yb, idesc, !first || k > 0, lead);
                }
            }
            mma_commit(&odone[st], lead);
            if (last) {
                mma_commit(&ofull[ob], lead);
                ++fl;
            }
        }
    } else if (MODE == kLse && warp >= 12) {
        const int set = (warp - 12) / S::kDzSet, quad = warp & 3, part = (warp - 12) % S::kDzSet >> 2;  // its 32 rows and 64 columns
        float c = a.ctemp, run_m = -INFINITY, run_s = 0.f;
        int he = 0, we_next = SPLIT && w.left ? __ldg(&a.wexp[w.y >> 1]) : 0;
        for (; w.left; ++g) {
            const int64_t row = (int64_t)w.x * 128 + quad * 32 + lane;
            if (w.y == w.y0) {
                run_m = -INFINITY;
                run_s = 0.f;
                if (SPLIT) he = row < a.X ? __ldg(&a.row_exp[row]) : 0;
            }
            // the tile's scale, held within fp32's range (what it makes of the scores is next to 0 there) and never 0: -inf stays -inf
            if (SPLIT) c = fmaxf(a.ctemp * exp2c(-he - we_next), 1e-37f);
            if ((g & 1) == set) {
                const uint32_t sb = g % NS;
                const int64_t left = a.Y - ((int64_t)w.y * BY + part * 64);
                ok = formed(g);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int ch = 0; ch < 2; ++ch) {
                    float v[32];
                    tm_ld32(tmem + ((uint32_t)(quad * 32) << 16) + sb * BY + part * 64 + ch * 32, v);
                    tm_wait_ld(v);
                    if (ch == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&pready[Pipe::turned(g).bar]);
                    }
                    take_scores(v, left - ch * 32, c, run_m, run_s);
                }
            }
            if (w.y + 1 == w.y1 && row < a.X)
                a.part[(row * a.slots + ((int)blockIdx.x - a.runs.first(w.x))) * S::kParts + set * (S::kParts / 2) + part] =
                    make_float2(run_m, run_s);
            step(w);
            if (SPLIT && w.left) we_next = __ldg(&a.wexp[w.y >> 1]);
        }
    } else if (MODE != kLse && warp >= 12) {
        const int set = (warp - 12) / S::kDzSet, quad = warp & 3, part = (warp - 12) % S::kDzSet >> 2;  // its 32 rows and 64 columns
        const int he = amax_exp(a.amax_h);
        // fetched while the warp works on the tile before; by asynchronous copies, which
        // hold no registers meanwhile
        auto fetch = [&](const Walk& t, Ahead& to) {
            if (!t.left) return;
            const int x32 = t.x * 4 + quad, y32 = t.y * (BY / 32) + part * 2;
            constexpr int kEach = COLS ? 16 : 8;  // lanes that copy each of the two or three rows of floats
            if (lane < (COLS ? 2 : 3) * kEach) {
                const int which = lane / kEach, at = lane % kEach * 4;
                const int64_t n = (int64_t)(COLS ? y32 : x32) * 32 + at;
                cp16((which == 0 ? to.nlse : which == 1 ? to.scale : to.scale + 32) + at, (which == 0 ? a.nlse : which == 1 ? a.scale : a.to_own) + n, true);
            }
            if (lane < 2) {
                const int nb = COLS ? y32 + lane : x32, vb = COLS ? x32 : y32 + lane;
                const bool have = nb < a.nblocks && vb < a.vblocks;
                cp16(&to.blk[lane], a.blocks + (have ? (int64_t)vb * a.nblocks + nb : 0), have);
                if (SPLIT && lane == 0) cp4(to.wexp, a.wexp + (COLS ? (DT == 64 ? t.x >> 1 : t.x) : t.y >> 1));
            }
        };
        if (set && w.left) step(w);
        int now = 0;
        fetch(w, ahead[warp - 12][0]);
        for (g = set; w.left; g += 2, now ^= 1) {
            const uint32_t sb = g % NS;
            const int64_t left = a.Y - ((int64_t)w.y * BY + part * 64);  // streamed rows from this warp's first column on
            const Ahead& my = ahead[warp - 12][now];
            const struct {
                int x32, y32;
            } at = {w.x * 4 + quad, w.y * (BY / 32) + part * 2};  // its 32-row blocks
            cp_wait();
            __syncwarp();
            step(w);
            if (w.left) step(w);
            fetch(w, ahead[warp - 12][now ^ 1]);
            const float c = SPLIT ? a.ctemp * exp2c(-he - my.wexp[0]) : a.ctemp;
            const float l = my.nlse[lane], r = my.scale[lane];  // of this lane's row (not COLS)
            ok = formed(g);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int ch = 0; ch < 2; ++ch) {
                const uint32_t t0 = tmem + ((uint32_t)(quad * 32) << 16) + sb * BY + part * 64 + ch * 32;
                float p[32];
                tm_ld32(t0, p);
                tm_wait_ld(p);
                if (COLS) {
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 l = *reinterpret_cast<const float4*>(my.nlse + ch * 32 + j);
                        const float4 r = *reinterpret_cast<const float4*>(my.scale + ch * 32 + j);
                        fma2(p[j], p[j + 1], c, c, l.x, l.y);
                        fma2(p[j + 2], p[j + 3], c, c, l.z, l.w);
#pragma unroll
                        for (int i = 0; i < 4; ++i) p[j + i] = ex2(p[j + i]);
                        mul2(p[j], p[j + 1], r.x, r.y);
                        mul2(p[j + 2], p[j + 3], r.z, r.w);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        fma2(p[j], p[j + 1], c, c, l, l);
                        p[j] = ex2(p[j]);
                        p[j + 1] = ex2(p[j + 1]);
                        mul2(p[j], p[j + 1], r, r);
                    }
                    if (left < ch * 32 + 32) {  // table rows past the last have no dz
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (ch * 32 + j >= left) p[j] = 0.f;
                    }
                }
                uint32_t q[16];
                pack32(p, q, SPLIT ? 0 : a.fmt);
                tm_st16(t0, q);
                if (SPLIT) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float2 h = unpack_f16(q[j]);
                        q[j] = pack16(p[2 * j] - h.x, p[2 * j + 1] - h.y, 0);
                    }
                    tm_st16(t0 + 16, q);
                }
                const uint4 b = my.blk[ch];
                if (b.x) {
                    tm_wait_st();
                    put_targets<SPLIT, COLS>(a, t0, b, COLS ? at.y32 + ch : at.x32, COLS ? at.x32 : at.y32 + ch, COLS ? 1.f : my.scale[32 + lane]);
                }
            }
            tm_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&pready[Pipe::turned(g).bar]);
        }
    } else if (MODE != kLse && warp >= 4) {
        const int half = warp >= 8, quad = warp & 3;
        const int eb = amax_exp(a.amax_z) + (COLS ? amax_exp(a.amax_h) : 0);
        constexpr int OC = DT / 64;  // 32-column chunks of this warp's half
        uint32_t fl = 0;
        bool first = true;
        while (ok && w.left) {
            const int64_t row = (int64_t)w.x * 128 + quad * 32 + lane;
            const uint32_t l0 = tmem + ((uint32_t)(quad * 32) << 16) + S::kOutCol + half * (DT / 2);
            const bool whole = w.y0 == 0 && w.y1 == a.runs.ytiles && !(MODE == kDhidden && a.low.K);
            const auto counts = [&] { return COLS || (row < a.X && __ldg(&a.scale[row]) != 0.f); };  // else dhidden is 0, whatever the table holds
            const auto scales = [&] {  // that the row's sums are still to be freed of; SPLIT dhidden: of its own only
                const int own = !COLS && a.zexp && row < a.X ? __ldg(&a.zexp[row]) : 0;
                return Pow2(SPLIT && !COLS ? -own : -eb - own);
            };
            float* part = a.partial + (((int64_t)blockIdx.x * 2 + !first) * 128 + quad * 32) * a.to.pp;
            auto put = [&](float(&v)[32], int col) {
                if (row - lane >= a.X || col >= a.D) return;
                if (!counts()) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0.f;
                }
                if (whole)
                    store_out(a.to, rows_out[warp - 4], 0, row - lane, col, a.X, a.D, v, scales());
                else
                    put_rows_f32(rows_out[warp - 4], v, reinterpret_cast<uint8_t*>(part + col), a.to.pp * 4, 32);
            };
            if (SPLIT) {
                float sum[OC][32];
#pragma unroll
                for (int ch = 0; ch < OC; ++ch)
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[ch][j] = 0.f;
                for (int f = w.y0; f < w.y1; f = (f | 1) + 1, ++fl) {
                    const uint32_t ob = fl % OB;
                    const Pow2 f1(COLS ? 0 : -eb - __ldg(&a.wexp[f >> 1]));
                    ok = head_wait(&ofull[ob], (fl / OB) & 1, a.wait_ns, gave_up);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int ch = 0; ch < 2 * OC; ++ch) {
                        float v[16];
#pragma unroll
                        for (int part = S::kOut / DT - 1; part >= 0; --part) {  // small products first
                            tm_read16(l0 + ob * S::kOut + part * DT + ch * 16, v);
#pragma unroll
                            for (int j = 0; j < 16; j += 2) {
                                if (!COLS && f1.b != 1.f) mul2(v[j], v[j + 1], f1.b, f1.b);
                                float &x = sum[ch / 2][(ch & 1) * 16 + j], &y = sum[ch / 2][(ch & 1) * 16 + j + 1];
                                if (COLS)
                                    add2(x, y, v[j], v[j + 1]);
                                else
                                    axpy2(x, y, v[j], v[j + 1], f1.a);  // exact products with powers of two
                            }
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&oempty[ob]);
                }
                if (!ok) break;
#pragma unroll
                for (int ch = 0; ch < OC; ++ch) put(sum[ch], half * (DT / 2) + ch * 32);
            } else {
                const uint32_t ob = fl % OB;
                ok = head_wait(&ofull[ob], (fl / OB) & 1, a.wait_ns, gave_up);
                if (!ok) break;
                ++fl;
                tc_fence_after();
                if (whole && a.to.vec && a.D == DT && a.to.type != TT_F32) {
                    // OUT is let go before anything is written: the next segment's product waits for it
                    const Pow2 sc = scales();
                    uint32_t q[OC][16];
#pragma unroll
                    for (int ch = 0; ch < OC; ++ch) {
                        float v[32];
                        tm_ld32(l0 + ob * S::kOut + ch * 32, v);
                        tm_wait_ld(v);
                        sc(v);
                        pack32(v, q[ch], a.fmt);
                        if (!counts()) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) q[ch][j] = 0;
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&oempty[ob]);
                    uint8_t* to = reinterpret_cast<uint8_t*>(static_cast<uint16_t*>(a.to.out) + (row - lane) * a.to.ldo + half * (DT / 2));
#pragma unroll
                    for (int ch = 0; ch < OC; ++ch) {
                        const uint4 mine[4] = {make_uint4(q[ch][0], q[ch][1], q[ch][2], q[ch][3]), make_uint4(q[ch][4], q[ch][5], q[ch][6], q[ch][7]),
                                               make_uint4(q[ch][8], q[ch][9], q[ch][10], q[ch][11]),
                                               make_uint4(q[ch][12], q[ch][13], q[ch][14], q[ch][15])};
                        put_rows(rows_out[warp - 4], mine, to + ch * 64, a.to.ldo * 2, a.X - (row - lane));
                    }
                } else {
#pragma unroll
                    for (int ch = 0; ch < OC; ++ch) {
                        float v[32];
                        tm_ld32(l0 + ob * S::kOut + ch * 32, v);
                        tm_wait_ld(v);
                        if (ch + 1 == OC) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&oempty[ob]);
                        }
                        put(v, half * (DT / 2) + ch * 32);
                    }
                }
            }
            first = false;
            w.left -= w.y1 - w.y0;
            ++w.x;
            w.y0 = 0;
            seg_end(w);
        }
    }
    if (!ok && lead) {
        *gave_up = 1;
        if (a.err) atomicOr(a.err, kErrTimeout);
    }
    __syncwarp();
    __syncthreads();
    if (*gave_up) {  // no copy and no MMA may still be running when the block ends
        if (threadIdx.x == 0) {
            for (uint32_t i = xu > S::XB ? xu - S::XB : 0; i < xu; ++i) head_drain(&xfull[i % S::XB], (i / S::XB) & 1);
            for (uint32_t i = g > S::kStages ? g - S::kStages : 0; i < g; ++i) head_drain(&yfull[i % S::kStages], (i / S::kStages) & 1);
        }
        if (lead && warp >= 1 && warp <= 3) {
            mma_commit(&drain[warp - 1], true);
            head_drain(&drain[warp - 1], 0);
        }
        __syncwarp();
        __syncthreads();
    }
    tc_fence_after();
    if (warp == 2) tc_dealloc(tmem, 512);
}

// Rows of an x that more than one run has tiles of: their segments summed in run order,
// 128 / gridDim.y rows per blockIdx.y.  blockIdx.x is the x, or (by_boundary: more x
// than runs) the boundary between two runs that lies in it; the first boundary inside
// an x takes it.
// With `low` every x is joined, were it from one run.  Sums are freed of the scales that
// amax_z, amax_y and (per row) zexp give.
__global__ void __launch_bounds__(128) k_head_join(Runs runs, int by_boundary, const float* partial, OutArgs to, int64_t X, int D,
                                                   const uint32_t* amax_z, const uint32_t* amax_y, const int* zexp, Residue low) {
    __shared__ int sh[4];
    if (threadIdx.x == 0) {
        int64_t x = blockIdx.x;
        bool split = true;
        int b = 0, last = 0, slot0 = 0;
        if (by_boundary) {
            const int64_t t = runs.begin(blockIdx.x + 1);
            x = t / runs.ytiles;
            split = x * runs.ytiles != t;
        }
        if (split) {
            b = runs.first(x);
            last = runs.last(x);
            split = (b != last || low.K) && (!by_boundary || b == (int)blockIdx.x);
            // in its first run x may come behind others (slot 1); every later run begins inside x
            slot0 = runs.begin(b) < x * runs.ytiles;
        }
        sh[0] = split ? (int)x : -1;
        sh[1] = b;
        sh[2] = last - b;
        sh[3] = slot0;
    }
    __syncthreads();
    const int64_t x = sh[0];
    if (x < 0) return;
    const int more = sh[2], per_row = (int)to.pp / 4, rows = 128 / per_row, span = 128 / gridDim.y;
    const int c = (int)threadIdx.x % per_row * 4, r0 = (int)threadIdx.x / per_row;
    if (r0 >= rows || c >= D) return;
    const int e = amax_exp(amax_z) + amax_exp(amax_y);
    const int64_t step = 256 * to.pp;
    for (int i = r0; i < span; i += rows) {
        const int r = blockIdx.y * span + i;
        if (x * 128 + r >= X) break;
        const Pow2 sc(-e - (zexp ? __ldg(&zexp[x * 128 + r]) : 0));
        const float* p = partial + ((int64_t)sh[1] * 256 + r) * to.pp + c;
        float4 s = *reinterpret_cast<const float4*>(p + sh[3] * 128 * to.pp);
#pragma unroll 4
        for (int k = 1; k <= more; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(p + k * step);
            s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
        }
        float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (low.K && c + j < D) v[j] += low(x * 128 + r, c + j);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c + j < D) store_one(to.out, (x * 128 + r) * to.ldo + c + j, sc(v[j]), to.type);
    }
}

}  // namespace ttemb
