// tt_head_fused.cuh -- the gradients of the vocabulary head for widths up to 128,
// dz kept on the chip.
//
//   dhidden[n] = sum_v dz[n, v] weight[v]        resident rows: hidden, streamed: weight
//   dweight[v] = sum_n dz[n, v] hidden[n]        resident rows: weight, streamed: hidden
//
// One kernel for both: a block holds 128 resident rows X and streams tiles of BY rows
// Y.  Per tile, S = X Y^T (tensor cores, K = D), eight warps turn S into dz (one
// exponential an element) and write it back to tensor memory in 16 bits, where it is
// the A operand of OUT += dz Y (K = BY); the same bytes of Y in shared memory are read
// K-major by the first product and MN-major by the second.  At these widths dz in
// memory would cost more than forming S twice: 6 bytes of traffic an element (written
// once, read twice) against 2 D FLOP and one exponential.
//
// S is double-buffered, and the MMA thread runs two tiles ahead with it, so that the
// tensor cores form S(i + 1) and OUT(i - 1) while the warps work on S(i).  X and OUT
// are double-buffered too (X but once for fp32 at D > 64, where shared memory is full),
// and eight further warps take OUT to memory, so units follow each other without a gap.
//
// SPLIT (fp32: every operand as f16 hi + lo): three products each; OUT covers one tile
// of Y at a time and its sums are kept in the storing warps' registers (k_head_gemm
// says why).
#pragma once

#include "tt_head.cuh"

namespace ttemb {

constexpr int kFusedThreads = 640;  // warp 0: TMA, 1: MMA, 2: tensor memory, 4..11: OUT, 12..19: dz

// A target's element of dz: lists by 32 x 32 block of (hidden row, table row).
struct __align__(16) TargetEntry {
    int next;   // next entry of the block's list, -1: none
    int at;     // (n & 31) | (v & 31) << 5
    float val;  // dz of the element, scaled like the others
    int pad;
};

struct FusedArgs {
    int64_t X, Y;   // resident and streamed rows
    int D;
    int xtiles, ytiles, splits;
    int64_t units;  // xtiles * splits
    int fmt;
    uint64_t wait_ns;
    int* err;
    const uint32_t* amax_h;  // power-of-two scales of hidden, weight, dz (null: none)
    const uint32_t* amax_w;
    const uint32_t* amax_z;
    float ctemp;             // log2(e) / T
    const float2* rowc;      // per hidden row (lse in log2 units, scale)
    const int* heads;        // [vblocks][nblocks] first entry of each block's list, -1: none
    const TargetEntry* ents;
    int nblocks, vblocks;
    OutArgs to;
};

template <int DT, bool SPLIT>
struct FusedShape {
    static constexpr int BY = SPLIT && DT == 128 ? 64 : 128;
    static constexpr int PC = SPLIT ? 2 : 1, DB = DT / 64;
    static constexpr int XB = SPLIT && DT == 128 ? 1 : 2;
    static constexpr int kStages = DT == 64 && !SPLIT ? 6 : 4;
    static constexpr uint32_t kXBlock = 128 * 128, kYBlock = BY * 128;  // 64 columns of a tile
    static constexpr uint32_t kX = PC * DB * kXBlock, kY = PC * DB * kYBlock;
    static constexpr size_t kSmem = (size_t)XB * kX + (size_t)kStages * kY + 1024;
    static constexpr uint32_t kOutCol = 256;  // tensor memory: S at 0 and BY, OUT at 256 and 256 + DT
};

// COLS: the streamed rows are hidden rows (dweight), so lse and scale go by column.
template <int DT, bool SPLIT, bool COLS>
__global__ void __launch_bounds__(kFusedThreads, 1)
    k_head_fused(const __grid_constant__ CUtensorMap mapX, const __grid_constant__ CUtensorMap mapY,
                 const __grid_constant__ FusedArgs a) {
    using S = FusedShape<DT, SPLIT>;
    constexpr int BY = S::BY, CH = BY / 64, kSegs = SPLIT ? 3 : 1;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t xfull[S::XB], xempty[S::XB], yfull[S::kStages], yempty[S::kStages];
    __shared__ uint64_t sfull[2], pready[2], pfree[2], ofull[2], oempty[2], drain;
    __shared__ float4 consts[COLS ? 8 : 1][CH * 16];  // per dz warp: (lse, scale) of its columns
    __shared__ uint32_t tmem_slot;
    __shared__ int gave_up_s;
    volatile int* gave_up = &gave_up_s;
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    const uint32_t ybase = base + S::XB * S::kX;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::XB; ++i) {
            mbar_init(&xfull[i], 1);
            mbar_init(&xempty[i], 1);
        }
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&yfull[i], 1);
            mbar_init(&yempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sfull[i], 1);
            mbar_init(&pready[i], 8);
            mbar_init(&pfree[i], 1);
            mbar_init(&ofull[i], 1);
            mbar_init(&oempty[i], 8);
        }
        mbar_init(&drain, 1);
        gave_up_s = 0;
    }
    if (warp == 2) tc_alloc(&tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    // The tiles of this block, in order: unit by unit, tile y of [y0, y1) of unit u.
    struct Walk {
        int64_t u;
        int x, split, y, y0, y1;
    };
    auto start = [&](Walk& w, int64_t u) {
        w.u = u;
        if (u >= a.units) return;
        w.split = (int)(u / a.xtiles);
        w.x = (int)(u - (int64_t)w.split * a.xtiles);
        w.y0 = w.y = (int)((int64_t)a.ytiles * w.split / a.splits);
        w.y1 = (int)((int64_t)a.ytiles * (w.split + 1) / a.splits);
    };
    auto step = [&](Walk& w) {
        if (++w.y == w.y1) start(w, w.u + gridDim.x);
    };
    Walk w;
    start(w, blockIdx.x);
    bool ok = true;
    uint32_t g = 0, xu = 0;  // tiles and units fed (TMA thread) or taken (the others)

    if (warp == 0) {
        if (lane == 0) {
            for (; w.u < a.units; step(w), ++g) {
                if (w.y == w.y0) {
                    const uint32_t b = xu % S::XB;
                    ok = head_wait(&xempty[b], ((xu / S::XB) & 1) ^ 1, a.wait_ns, gave_up);
                    if (!ok) break;
                    bulk_expect(&xfull[b], S::kX);
                    for (int i = 0; i < S::PC * S::DB; ++i)
                        tma_load3(base + b * S::kX + i * S::kXBlock, &mapX, (i % S::DB) * 64, w.x * 128, i / S::DB, &xfull[b]);
                    ++xu;
                }
                const uint32_t st = g % S::kStages;
                ok = head_wait(&yempty[st], ((g / S::kStages) & 1) ^ 1, a.wait_ns, gave_up);
                if (!ok) break;
                bulk_expect(&yfull[st], S::kY);
                for (int i = 0; i < S::PC * S::DB; ++i)
                    tma_load3(ybase + st * S::kY + i * S::kYBlock, &mapY, (i % S::DB) * 64, w.y * BY, i / S::DB, &yfull[st]);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t id_s = idesc_f16(128, BY, a.fmt, false, false), id_o = idesc_f16(128, DT, a.fmt, false, true);
            const int ksteps = (a.D + 15) / 16;
            uint32_t gs = 0, fl = 0;
            Walk ws = w;
            auto issue_s = [&]() {
                const uint32_t b = xu % S::XB, st = gs % S::kStages, sb = gs & 1;
                if (ws.y == ws.y0) {
                    ok = head_wait(&xfull[b], (xu / S::XB) & 1, a.wait_ns, gave_up);
                    if (!ok) return;
                }
                ok = head_wait(&yfull[st], (gs / S::kStages) & 1, a.wait_ns, gave_up) &&
                     head_wait(&pfree[sb], ((gs >> 1) & 1) ^ 1, a.wait_ns, gave_up);
                if (!ok) return;
                tc_fence_after();
                const uint32_t d = tmem + sb * BY;
#pragma unroll
                for (int seg = 0; seg < kSegs; ++seg) {
                    const uint32_t sx = base + b * S::kX + (SPLIT && seg == 0 ? S::DB * S::kXBlock : 0);
                    const uint32_t sy = ybase + st * S::kY + (SPLIT && seg == 1 ? S::DB * S::kYBlock : 0);
                    for (int k = 0; k < ksteps; ++k)
                        mma_f16(d, desc_sw128(sx + (k >> 2) * S::kXBlock + (k & 3) * 32, false, 0),
                                desc_sw128(sy + (k >> 2) * S::kYBlock + (k & 3) * 32, false, 0), id_s, seg > 0 || k > 0);
                }
                tc_commit(&sfull[sb]);
                ++gs;
                if (ws.y + 1 == ws.y1) {
                    tc_commit(&xempty[b]);  // nothing but S reads X
                    ++xu;
                }
                step(ws);
            };
            if (ws.u < a.units) issue_s();
            if (ok && ws.u < a.units) issue_s();
            for (; ok && w.u < a.units; step(w), ++g) {
                const uint32_t st = g % S::kStages, sb = g & 1, ob = fl & 1;
                const bool first = SPLIT || w.y == w.y0, last = SPLIT || w.y + 1 == w.y1;
                ok = head_wait(&pready[sb], (g >> 1) & 1, a.wait_ns, gave_up);
                if (ok && first) ok = head_wait(&oempty[ob], ((fl >> 1) & 1) ^ 1, a.wait_ns, gave_up);
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = tmem + S::kOutCol + ob * DT, p = tmem + sb * BY;
#pragma unroll
                for (int seg = 0; seg < kSegs; ++seg) {
                    const uint32_t sy = ybase + st * S::kY + (SPLIT && seg == 1 ? S::DB * S::kYBlock : 0);
#pragma unroll
                    for (int k = 0; k < BY / 16; ++k)
                        mma_f16_ta(d, p + (k >> 1) * 32 + (k & 1) * 8 + (SPLIT && seg == 0 ? 16 : 0),
                                   desc_sw128(sy + k * 2048, true, S::kYBlock), id_o, !first || seg > 0 || k > 0);
                }
                tc_commit(&yempty[st]);
                tc_commit(&pfree[sb]);
                if (last) {
                    tc_commit(&ofull[ob]);
                    ++fl;
                }
                if (ws.u < a.units) issue_s();
            }
        }
    } else if (warp >= 12) {
        const int half = warp >= 16, quad = warp & 3;
        const float c = a.ctemp * exp2i(-amax_exp(a.amax_h)) * exp2i(-amax_exp(a.amax_w));
        float2 rc = make_float2(0.f, 0.f);
        for (; w.u < a.units; step(w), ++g) {
            const uint32_t sb = g & 1;
            const int64_t x0 = (int64_t)w.x * 128 + quad * 32, y0 = (int64_t)w.y * BY + half * (BY / 2);
            int head[CH];
#pragma unroll
            for (int ch = 0; ch < CH; ++ch) {
                const int64_t xb = x0 >> 5, yb = (y0 >> 5) + ch, nb = COLS ? yb : xb, vb = COLS ? xb : yb;
                head[ch] = nb < a.nblocks && vb < a.vblocks ? __ldg(&a.heads[vb * a.nblocks + nb]) : -1;
            }
            if (COLS) {
                __syncwarp();
#pragma unroll
                for (int ch = 0; ch < CH; ++ch) {
                    const int64_t n = y0 + ch * 32 + lane;
                    reinterpret_cast<float2*>(consts[warp - 12])[ch * 32 + lane] = n < a.Y ? __ldg(&a.rowc[n]) : make_float2(0.f, 0.f);
                }
                __syncwarp();
            } else if (w.y == w.y0) {
                rc = x0 + lane < a.X ? __ldg(&a.rowc[x0 + lane]) : make_float2(0.f, 0.f);
            }
            ok = __all_sync(0xffffffffu, head_wait(&sfull[sb], (g >> 1) & 1, a.wait_ns, gave_up));
            if (!ok) break;
            tc_fence_after();
            const uint32_t t0 = tmem + ((uint32_t)(quad * 32) << 16) + sb * BY + half * (BY / 2);
            float v[2][32];
            tm_ld32(t0, v[0]);
            tm_wait_ld(v[0]);
#pragma unroll
            for (int ch = 0; ch < CH; ++ch) {
                if (ch + 1 < CH) tm_ld32(t0 + (ch + 1) * 32, v[(ch + 1) & 1]);
                float(&p)[32] = v[ch & 1];
                if (COLS) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float4 k = consts[warp - 12][ch * 16 + j];  // columns 2 j and 2 j + 1
                        p[2 * j] = k.y * ex2(fmaf(p[2 * j], c, -k.x));
                        p[2 * j + 1] = k.w * ex2(fmaf(p[2 * j + 1], c, -k.z));
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) p[j] = rc.y * ex2(fmaf(p[j], c, -rc.x));
                    const int64_t left = a.Y - (y0 + ch * 32);  // table rows past the last have no dz
                    if (left < 32) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (j >= left) p[j] = 0.f;
                    }
                }
                for (int e = head[ch]; e >= 0;) {
                    const int4 t = __ldg(reinterpret_cast<const int4*>(a.ents + e));
                    const int tn = t.y & 31, tv = t.y >> 5, tl = COLS ? tv : tn, tc = COLS ? tn : tv;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j == tc && lane == tl) p[j] = __int_as_float(t.z);
                    e = t.x;
                }
                uint32_t q[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) q[j] = pack16(p[2 * j], p[2 * j + 1], a.fmt);
                tm_st16(t0 + ch * 32, q);
                if (SPLIT) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float2 h = unpack_f16(q[j]);
                        q[j] = pack16(p[2 * j] - h.x, p[2 * j + 1] - h.y, 0);
                    }
                    tm_st16(t0 + ch * 32 + 16, q);
                }
                if (ch + 1 < CH) tm_wait_ld(v[(ch + 1) & 1]);
            }
            tm_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&pready[sb]);
        }
    } else if (warp >= 4) {
        const int half = warp >= 8, quad = warp & 3;
        const float s1 = exp2i(-amax_exp(a.amax_z)), s2 = exp2i(-amax_exp(COLS ? a.amax_h : a.amax_w));
        constexpr int OC = DT / 64;  // 32-column chunks of this warp's half
        uint32_t fl = 0;
        for (; w.u < a.units; start(w, w.u + gridDim.x)) {
            float sum[OC][32];
            const int flushes = SPLIT ? w.y1 - w.y0 : 1;
            for (int f = 0; f < flushes; ++f, ++fl) {
                const uint32_t ob = fl & 1;
                ok = __all_sync(0xffffffffu, head_wait(&ofull[ob], (fl >> 1) & 1, a.wait_ns, gave_up));
                if (!ok) break;
                tc_fence_after();
                const uint32_t t0 = tmem + ((uint32_t)(quad * 32) << 16) + S::kOutCol + ob * DT + half * (DT / 2);
#pragma unroll
                for (int ch = 0; ch < OC; ++ch) {
                    float v[32];
                    tm_ld32(t0 + ch * 32, v);
                    tm_wait_ld(v);
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[ch][j] = f == 0 ? v[j] : sum[ch][j] + v[j];
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&oempty[ob]);
            }
            if (!ok) break;
            const int64_t row = (int64_t)w.x * 128 + quad * 32 + lane;
#pragma unroll
            for (int ch = 0; ch < OC; ++ch) {
                const int64_t col = half * (DT / 2) + ch * 32;
                if (row < a.X && col < a.D) store_out(a.to, w.split, row, col, a.X, a.D, sum[ch], s1, s2);
            }
        }
    }
    if (!ok) {
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
        if (threadIdx.x == 32) {
            tc_commit(&drain);
            head_drain(&drain, 0);
        }
        __syncwarp();
        __syncthreads();
    }
    tc_fence_after();
    if (warp == 2) tc_dealloc(tmem, 512);
}

}  // namespace ttemb
