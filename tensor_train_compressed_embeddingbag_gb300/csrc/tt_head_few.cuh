// tt_head_few.cuh -- scores of up to eight hidden rows at a time: the single tokens of a
// serving step and small batches.
//
// With so few rows a pass over the table is bound by reading it (2 N FLOP per element
// against 2 or 4 bytes), so the table is read once, as it is, straight into registers:
// no copies in 16-bit pieces, and no 128-row tiles that are mostly padding.  The products
// run on the warp-level tensor cores with the table's rows as the long side
// (mma.sync: 16 table rows x 8 hidden rows); fp32 as TF32 hi and lo parts, hi hi + hi lo +
// lo hi, split on the fly (a step whose numbers are not all finite, or round to infinity, in
// a slower way that keeps them what they are).  The order of k is free as long as both operands use the same,
// so a thread's part of a table row is 16 bytes in one load (four, where rows do not begin
// on 16-byte boundaries), and the hidden rows lie in shared
// memory as the fragments want them.  A warp takes 32 table rows at a time; where there
// are too few of them, warps share a row's columns.  Sums over 64 bytes x 2 of a row are
// added up in fp32 registers.  Each lane keeps the running maximum and sum of the table
// row it holds; lanes, warps and blocks are joined at the end.
//
// Measured: bf16 4 x 131072 x 4096, 1.07 GB, 190 us (5.6 TB/s); fp32 8 x 131072 x 1024,
// 0.54 GB, 99 us (5.4 TB/s).  A step's loads go to the registers of the one before, which
// bounds the bytes in flight at 16 warps to an SM; loads to shared memory are not tried.
#pragma once

#include <type_traits>

#include "tt_head.cuh"

namespace ttemb {

constexpr int kFewThreads = 256, kFewWarps = 8, kFewRows = 32;
constexpr int kFewStep = 2;                   // chunks (64 bytes of a row) loaded at a time
constexpr size_t kFewSmem = 200 * 1024;      // of them in shared memory, at most

struct FewArgs {
    const void* h;
    const void* w;
    int64_t ldh, ldw, V;
    int N, D;
    int chunks;   // 64-byte pieces of a table row
    int ksplit;   // warps that share a table tile
    float c;      // log2(e) / T
    float2* part; // [N][gridDim.x] (maximum in log2 units, sum)
};

__device__ __forceinline__ void mma_few(float* d, const uint32_t* a, const uint32_t* b, const uint32_t* a8, int type) {
    // a: two registers of rows g, a8: of rows g + 8
    if (type == TT_BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a8[0]), "r"(a[1]), "r"(a8[1]), "r"(b[0]), "r"(b[1]));
    else if (type == TT_F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a8[0]), "r"(a[1]), "r"(a8[1]), "r"(b[0]), "r"(b[1]));
    else
        asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a8[0]), "r"(a[1]), "r"(a8[1]), "r"(b[0]), "r"(b[1]));
}

// x as its TF32 part and the rest (exact), both rounded to nearest by adding half a unit:
// the tensor core cuts what TF32 does not hold.  Not for what that carries out of the finite
// numbers, infinities and NaN.
__device__ __forceinline__ void few_split(uint32_t& x, uint32_t& lo) {
    const uint32_t hi = (x + 0x1000u) & 0xFFFFE000u;
    lo = __float_as_uint(__uint_as_float(x) - __uint_as_float(hi)) + 0x1000u;
    x = hi;
}
// The same for any x (a quarter of the rate).  The rounding saturates: an infinity becomes the
// largest number and an infinite rest, which meets the other operand's first part once, with
// its sign; rounded to an infinity its rest would be NaN.  NaN stays NaN.
__device__ __forceinline__ void few_split_any(uint32_t& x, uint32_t& lo) {
    uint32_t hi;
    asm("cvt.rna.satfinite.tf32.f32 %0, %1;" : "=r"(hi) : "f"(__uint_as_float(x)));
    lo = __float_as_uint(__uint_as_float(x) - __uint_as_float(hi)) + 0x1000u;
    x = hi;
}
constexpr float kFewMost = 3.401992698887923e38f;  // the largest number that few_split rounds down
__device__ __forceinline__ float max_abs(float m, uint32_t a, uint32_t b) {  // NaN if any is
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(__uint_as_float(a))), "f"(fabsf(__uint_as_float(b))));
    return r;
}

template <class T, int TYPE, bool WIDE>  // WIDE: table rows begin on 16-byte boundaries, else on 4-byte ones
__global__ void __launch_bounds__(kFewThreads, 2) k_head_few(const __grid_constant__ FewArgs a) {
    constexpr int E = 16 / sizeof(T), C = kFewStep;
    constexpr bool TWO = TYPE == TT_F32;  // hi and lo parts
    extern __shared__ uint4 xs[];         // [chunk][32 lanes]
    __shared__ float red[kFewWarps][kFewRows * 8];
    __shared__ float2 parts[kFewWarps][8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;

    float hmax = 0.f;
    for (int i = threadIdx.x; i < a.chunks * 32; i += kFewThreads) {
        const int l = i & 31, m = l >> 2, d0 = ((i >> 5) * 4 + (l & 3)) * E;
        __align__(16) T y[E];
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = m < a.N && d0 + e < a.D ? static_cast<const T*>(a.h)[m * a.ldh + d0 + e] : T(0.f);
        const uint4 u = *reinterpret_cast<uint4*>(y);
        xs[i] = u;
        if (TWO) hmax = max_abs(max_abs(hmax, u.x, u.y), u.z, u.w);
    }
    const bool any_hidden = __syncthreads_or(TWO && !(hmax <= kFewMost));  // hidden rows that few_split is not for

    const int tiles_per_block = kFewWarps / a.ksplit, sub = warp / a.ksplit, ks = warp - sub * a.ksplit;
    const int steps = (a.chunks + C - 1) / C, jb = steps * ks / a.ksplit, je = steps * (ks + 1) / a.ksplit;
    const int64_t ntiles = (a.V + kFewRows - 1) / kFewRows, rounds = (ntiles + tiles_per_block - 1) / tiles_per_block;
    const int64_t pitch = a.ldw * (int64_t)sizeof(T);
    const int row_bytes = a.D * (int)sizeof(T);

    // the next step to load: round lr, step lj; table rows tile * 32 + {0, 8, 16, 24} + g
    // (rows past V read row V - 1)
    int64_t lr = blockIdx.x;
    int lj = jb;
    const uint8_t* pr[4];
    auto at_tile = [&]() {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            int64_t v = (lr * tiles_per_block + sub) * kFewRows + r * 8 + g;
            v = v < a.V ? v : a.V - 1;
            pr[r] = static_cast<const uint8_t*>(a.w) + v * pitch;
        }
    };
    at_tile();
    auto load = [&](uint4 (&q)[4][C]) {
        if (lr >= rounds) return;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int at = ((lj * C + i) * 4 + t) * 16;
#pragma unroll
            for (int r = 0; r < 4; ++r) {  // past the row's end: 0, so that nothing not finite meets hidden's 0
                if (WIDE) {
                    q[r][i] = at < row_bytes ? __ldcs(reinterpret_cast<const uint4*>(pr[r] + at)) : make_uint4(0, 0, 0, 0);
                } else {
                    const uint32_t* p = reinterpret_cast<const uint32_t*>(pr[r] + at);
                    q[r][i] = make_uint4(at < row_bytes ? __ldg(p) : 0, at + 4 < row_bytes ? __ldg(p + 1) : 0,
                                         at + 8 < row_bytes ? __ldg(p + 2) : 0, at + 12 < row_bytes ? __ldg(p + 3) : 0);
                }
            }
        }
        if (++lj == je) {
            lj = jb;
            lr += gridDim.x;
            if (lr < rounds) at_tile();
        }
    };
    constexpr int U = 2;
    uint4 q[U][4][C];
#pragma unroll
    for (int i = 0; i < U; ++i) load(q[i]);

    float tot[2][4], run_m[8], run_s[8];
#pragma unroll
    for (int m = 0; m < 8; ++m) {
        run_m[m] = -INFINITY;
        run_s[m] = tot[m >> 2][m & 3] = 0.f;
    }
    int64_t rd = blockIdx.x;
    int j = jb;
    while (rd < rounds) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (rd >= rounds) break;
            float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            auto products = [&](auto any) {
                auto split = [](uint32_t& x, uint32_t& lo) { decltype(any)::value ? few_split_any(x, lo) : few_split(x, lo); };
#pragma unroll
                for (int ch = 0; ch < C; ++ch) {
                    const int c = j * C + ch;
                    if (c >= a.chunks) break;
                    const uint4 bv = xs[c * 32 + lane];
                    uint32_t b[4] = {bv.x, bv.y, bv.z, bv.w}, bl[4];
                    if (TWO)
#pragma unroll
                        for (int e = 0; e < 4; ++e) split(b[e], bl[e]);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint4 u0 = q[i][2 * r][ch], u8 = q[i][2 * r + 1][ch];
                        uint32_t f0[4] = {u0.x, u0.y, u0.z, u0.w}, f8[4] = {u8.x, u8.y, u8.z, u8.w}, l0[4], l8[4];
                        if (TWO)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                split(f0[e], l0[e]);
                                split(f8[e], l8[e]);
                            }
#pragma unroll
                        for (int k = 0; k < 4; k += 2) {
                            if (TWO) {
                                mma_few(acc[r], l0 + k, b + k, l8 + k, TYPE);
                                mma_few(acc[r], f0 + k, bl + k, f8 + k, TYPE);
                            }
                            mma_few(acc[r], f0 + k, b + k, f8 + k, TYPE);
                        }
                    }
                }
            };
            if (TWO) {
                float m = 0.f;
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int ch = 0; ch < C; ++ch) m = max_abs(max_abs(m, q[i][r][ch].x, q[i][r][ch].y), q[i][r][ch].z, q[i][r][ch].w);
                if (__any_sync(0xffffffffu, any_hidden || !(m <= kFewMost)))
                    products(std::true_type());
                else
                    products(std::false_type());
            } else {
                products(std::false_type());
            }
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) tot[r][e] += acc[r][e];
            load(q[i]);
            if (++j < je) continue;
            // the tile's scores through shared memory: a lane takes one table row; warps
            // that share the tile take hidden rows in turn
            const int64_t v = (rd * tiles_per_block + sub) * kFewRows + lane;
            if (a.ksplit > 1)
                __syncthreads();
            else
                __syncwarp();
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    red[warp][(2 * t + (e & 1)) * kFewRows + r * 16 + (e >> 1) * 8 + g] = tot[r][e];
                    tot[r][e] = 0.f;
                }
            if (a.ksplit > 1)
                __syncthreads();
            else
                __syncwarp();
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                if (m >= a.N || (m & (a.ksplit - 1)) != ks || v >= a.V) continue;
                float z = 0.f;
                for (int k = 0; k < a.ksplit; ++k) z += red[sub * a.ksplit + k][m * kFewRows + lane];
                z *= a.c;
                const float mn = fmaxf(run_m[m], z), b = mn == -INFINITY ? 0.f : mn;
                run_s[m] = run_s[m] * ex2(run_m[m] - b) + ex2(z - b);
                run_m[m] = mn;
            }
            j = jb;
            rd += gridDim.x;
        }
    }
    // lanes, then warps
#pragma unroll
    for (int m = 0; m < 8; ++m) {
        float x = run_m[m];
#pragma unroll
        for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
        const float b = x == -INFINITY ? 0.f : x;
        float s = run_s[m] * ex2(run_m[m] - b);
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) parts[warp][m] = make_float2(x, s);
    }
    __syncthreads();
    if (threadIdx.x < a.N) {
        float x = -INFINITY, s = 0.f;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) x = fmaxf(x, parts[w][threadIdx.x].x);
        const float b = x == -INFINITY ? 0.f : x;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) s += parts[w][threadIdx.x].y * ex2(parts[w][threadIdx.x].x - b);
        a.part[(int64_t)threadIdx.x * gridDim.x + blockIdx.x] = make_float2(x, s);
    }
}

}  // namespace ttemb
