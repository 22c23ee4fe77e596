// tt_q4.cu -- scores of a few rows against a table held in 4 bits (serving):
//
//   out[m, v] = sum_j scale[v, j] sum_{d in group j} (code[v, d] - 8) x[m, d]
//
// Codes are 4-bit, two to a byte (the even column in the low half), rows padded to a
// multiple of 32 columns; one bf16 scale per group of 32, 64 or 128 columns.
//
// A call reads half a byte per weight and multiplies it by the few rows of x, so reading
// the table is its floor.  What the kernel does per weight has to fit beside the loads:
// codes become f16 two at a time (an OR puts two codes into the mantissas of 1024 or, at
// the next higher nibble, of 1024 in steps of 16; one packed operation leaves code - 8,
// exactly: the conversion of Y. J. Kim et al., "Who Says Elephants Can't Run: Bringing Large
// Scale MoE Models into Cloud Scale Production", 2022), and the products run on the
// warp-level tensor cores (mma.sync.m16n8k16: 16 table rows x 8 rows of x), fp32
// accumulation per group, one fp32 multiply-add by the group's scale into the running sum.
//
// x in f16: f16 rows as they are; bf16 and fp32 rows times a power of two that puts the
// row's largest magnitude near 2^14.  A bf16 value is then an f16 value (its 8 bits fit;
// values below 2^-31 of the row's largest lose bits, by at most 2^-39 of it), an fp32
// value the sum of two (hi + lo, 22 bits), one MMA each.  So the products of what x enters
// as are exact.
//
// The order of k inside a group is free as long as both operands use the same: a thread's
// share of a group is one contiguous load of group / 8 bytes per table row, and x lies in
// shared memory in the order in which the fragments want it.  A warp takes 32 table rows
// at a time and keeps the loads of the next groups, of this tile or the next, in flight.
//
// Measured: 1 x 131072 x 4096, groups of 128, bf16 x: 277 MB in 63 us (4.4 TB/s; floor 41);
// 8 x 1,000,000 x 64, groups of 32, fp32 x: 68 MB in 19.7 us (floor 10).  The ALU that
// turns codes into f16 is 46 and 48% busy, half of all issue slots go, and a warp waits
// mostly on its own last instruction: neither bound is reached.  The table's bytes go to
// registers (118 to 125 a thread at 16 warps to an SM), which holds how many are in flight;
// copies to shared memory, which hold none, are not tried.  Codes as
// f16 subnormals would spare the OR, but lose the scale's low bits.
#include <type_traits>

#include "tt_head.cuh"

namespace ttemb {

constexpr int kQ4Threads = 256;
constexpr int kQ4Warps = kQ4Threads / 32;
constexpr int kQ4Rows = 32;                 // table rows per warp (two MMA row tiles)
constexpr int kQ4SmemBytes = 96 * 1024;     // x fragments of one launch

struct Q4Args {
    const void* x;
    int64_t ldx;
    int m0, M;              // rows of x of this launch: [m0, m0 + M)
    int D;
    const uint8_t* packed;  // [V][pitch]
    int64_t pitch;          // bytes per row
    const __nv_bfloat16* scales;  // [V][groups]
    int groups;
    int g0, g1;             // groups of this launch
    int64_t V;
    float* out;             // [.][V]
    int accumulate;
    int ksplit;             // warps that share the groups of a table tile
    int vec;                // rows of x are 16-byte aligned
    uint32_t thousand;      // 0x64006400, not a literal in the kernel (and_or)
};

// (w & mask) | bits in one instruction, given that only one of the two is a literal.
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t bits) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(bits));
    return r;
}

// (code - 8) of columns i and i + 4 of the eight codes of w, i = 0 .. 3.  thousand: the
// bits of two f16 1024s.
__device__ __forceinline__ void q4_pairs(uint32_t w, uint32_t thousand, uint32_t (&f)[4]) {
    const uint32_t h = w >> 8;
    const uint32_t c0 = and_or(w, 0x000F000Fu, thousand), c1 = and_or(w, 0x00F000F0u, thousand);  // 1024 + q, 1024 + 16 q
    const uint32_t c2 = and_or(h, 0x000F000Fu, thousand), c3 = and_or(h, 0x00F000F0u, thousand);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(f[0]) : "r"(c0), "r"(0x64086408u));                          // - 1032
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(f[1]) : "r"(c1), "r"(0x2C002C00u), "r"(0xD480D480u));    // / 16 - 72
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(f[2]) : "r"(c2), "r"(0x64086408u));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(f[3]) : "r"(c3), "r"(0x2C002C00u), "r"(0xD480D480u));
}

__device__ __forceinline__ void mma16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int W>
__device__ __forceinline__ void q4_load(const uint8_t* p, uint32_t (&q)[W]) {
    if constexpr (W == 4) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
        q[0] = u.x;
        q[1] = u.y;
        q[2] = u.z;
        q[3] = u.w;
    } else if constexpr (W == 2) {
        const uint2 u = __ldcs(reinterpret_cast<const uint2*>(p));
        q[0] = u.x;
        q[1] = u.y;
    } else {
        q[0] = __ldcs(reinterpret_cast<const uint32_t*>(p));
    }
}

// W = G / 32 words of 8 codes per thread, table row and group.  Shared memory:
// x as [group][word][piece][n tile][32 lanes] x 16 bytes: lane (g, t) of an MMA (g =
// lane / 4 the row of x, t = lane % 4) finds there x of the 8 columns that thread t
// holds in that word, in the order 0 4 1 5 2 6 3 7 of its nibbles.
template <class T, int G, int NT>
__global__ void __launch_bounds__(kQ4Threads, 2) k_q4_matvec(const __grid_constant__ Q4Args a) {
    constexpr int W = G / 32, P = sizeof(T) == 4 ? 2 : 1;
    extern __shared__ uint4 xs[];
    __shared__ float red[kQ4Warps][kQ4Rows * 8];  // one n tile at a time
    __shared__ float up[NT * 8], down[NT * 8];    // a row's power of two, and its inverse
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int ng = a.g1 - a.g0;

    const T* x = static_cast<const T*>(a.x) + (int64_t)a.m0 * a.ldx;
    for (int m = warp; m < NT * 8; m += kQ4Warps) {
        uint32_t most = 0;
        if (sizeof(T) != 2 || !std::is_same<T, __half>::value)
            if (m < a.M)
#pragma unroll 16
                for (int d = a.g0 * G + lane; d < min(a.g1 * G, a.D); d += 32) {
                    const uint32_t b = __float_as_uint(to_f32(x[m * a.ldx + d])) & 0x7FFFFFFFu;
                    if (b < 0x7F800000u) most = max(most, b);
                }
        const int e = scale_exp(__reduce_max_sync(0xffffffffu, most));
        if (lane == 0) {
            up[m] = exp2i(e);
            down[m] = exp2i(-e);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < ng * W * NT * 32; i += kQ4Threads) {
        const int l = i & 31, rest = i >> 5;
        const int nt = rest % NT, w = rest / NT % W, j = rest / NT / W;
        const int m = nt * 8 + (l >> 2), d0 = (a.g0 + j) * G + (l & 3) * (G / 4) + w * 8;
        uint16_t u[P][8];
        __align__(16) T y[8];
        const bool all = m < a.M && d0 + 8 <= a.D && a.vec;
        if (all)
#pragma unroll
            for (int e = 0; e < (int)sizeof(T) / 2; ++e)
                reinterpret_cast<uint4*>(y)[e] = __ldg(reinterpret_cast<const uint4*>(x + m * a.ldx + d0) + e);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int k = (e >> 1) + (e & 1) * 4;
            const float v = (all ? to_f32(y[k]) : (m < a.M && d0 + k < a.D ? to_f32(x[m * a.ldx + d0 + k]) : 0.f)) * up[m];
            if (P == 2) {
                const uint32_t hi = pack_hi(v, 0.f);
                u[0][e] = (uint16_t)hi;
                u[P - 1][e] = __half_as_ushort(__float2half_rn(v - unpack_f16(hi).x));
            } else {
                u[0][e] = __half_as_ushort(__float2half_rn(v));
            }
        }
#pragma unroll
        for (int p = 0; p < P; ++p) xs[(((j * W + w) * P + p) * NT + nt) * 32 + l] = *reinterpret_cast<uint4*>(u[p]);
    }
    __syncthreads();

    const int tiles_per_block = kQ4Warps / a.ksplit;
    const int sub = warp / a.ksplit, ks = warp - sub * a.ksplit;
    const int jb = ng * ks / a.ksplit, je = ng * (ks + 1) / a.ksplit;
    const int64_t ntiles = (a.V + kQ4Rows - 1) / kQ4Rows;
    const int64_t rounds = (ntiles + tiles_per_block - 1) / tiles_per_block;

    // the next group to load: round lr, group lj; four table rows per thread, tile * 32 +
    // {0, 8, 16, 24} + g (rows past V read row V - 1)
    int64_t lr = blockIdx.x;
    int lj = jb;
    const uint8_t* pr[4];
    const __nv_bfloat16* sr[4];
    auto at_tile = [&]() {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            int64_t v = (lr * tiles_per_block + sub) * kQ4Rows + r * 8 + g;
            v = v < a.V ? v : a.V - 1;
            pr[r] = a.packed + v * a.pitch;
            sr[r] = a.scales + v * a.groups;
        }
    };
    at_tile();
    auto load = [&](uint32_t (&q)[4][W], uint32_t (&s)[4]) {
        if (lr >= rounds) return;
        // a share past the row's end: any codes will do, x is 0 there
        int at = (a.g0 + lj) * (G / 2) + t * (G / 8);
        at = at < (int)a.pitch ? at : 0;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            q4_load<W>(pr[r] + at, q[r]);
            s[r] = *reinterpret_cast<const uint16_t*>(sr[r] + a.g0 + lj);
        }
        if (++lj == je) {
            lj = jb;
            lr += gridDim.x;
            if (lr < rounds) at_tile();
        }
    };
    constexpr int U = (W == 4 ? 2 : 4) / (NT == 4 ? 2 : 1);  // groups in flight, as registers allow
    uint32_t q[U][4][W], s[U][4];
#pragma unroll
    for (int i = 0; i < U; ++i) load(q[i], s[i]);

    float tot[2][NT][4];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) tot[r][n][e] = 0.f;
    int64_t rd = blockIdx.x;
    int j = jb;
    while (rd < rounds) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (rd >= rounds) break;
            float acc[2][NT][4];
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[r][n][e] = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                uint32_t f[4][4];
#pragma unroll
                for (int r = 0; r < 4; ++r) q4_pairs(q[i][r][w], a.thousand, f[r]);
#pragma unroll
                for (int p = P - 1; p >= 0; --p)  // small products first
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint4 b = xs[(((j * W + w) * P + p) * NT + n) * 32 + lane];
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            mma16816(acc[r][n], f[2 * r][0], f[2 * r + 1][0], f[2 * r][1], f[2 * r + 1][1], b.x, b.y);
                            mma16816(acc[r][n], f[2 * r][2], f[2 * r + 1][2], f[2 * r][3], f[2 * r + 1][3], b.z, b.w);
                        }
                    }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) tot[r][n][e] = fmaf(__uint_as_float(s[i][2 * r + (e >> 1)] << 16), acc[r][n][e], tot[r][n][e]);
            load(q[i], s[i]);
            if (++j < je) continue;
            // the tile's last group: element (row, m) of n tile n is tot[..][n][..]
            const int64_t v0 = (rd * tiles_per_block + sub) * kQ4Rows;
            if (a.ksplit == 1) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int m = n * 8 + 2 * t + e;
                        if (m >= a.M) continue;
                        float* o = a.out + (int64_t)(a.m0 + m) * a.V + v0 + g;
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            if (v0 + r * 8 + g >= a.V) continue;
                            const float y = tot[r >> 1][n][(r & 1) * 2 + e] * down[m];
                            o[r * 8] = a.accumulate ? o[r * 8] + y : y;
                        }
                    }
            } else {  // joined with the other warps of the tile
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (n * 8 >= a.M) break;
                    __syncthreads();
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int e = 0; e < 4; ++e) red[warp][(2 * t + (e & 1)) * kQ4Rows + r * 16 + (e >> 1) * 8 + g] = tot[r][n][e];
                    __syncthreads();
                    const int64_t v = v0 + lane;
                    for (int m = ks; m < 8; m += a.ksplit) {
                        if (n * 8 + m >= a.M || v >= a.V) continue;
                        float sum = 0.f;
                        for (int k = 0; k < a.ksplit; ++k) sum += red[sub * a.ksplit + k][m * kQ4Rows + lane];
                        sum *= down[n * 8 + m];
                        float* o = a.out + (int64_t)(a.m0 + n * 8 + m) * a.V + v;
                        *o = a.accumulate ? *o + sum : sum;
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) tot[r][n][e] = 0.f;
            j = jb;
            rd += gridDim.x;
        }
    }
}

// Codes and scales of a table: per group, scale = bf16(max |w| / 7), code = w / scale
// rounded to nearest (ties to even), held within [-8, 7], plus 8.  A group that holds an
// infinity has an infinite scale, one with a NaN a scale of NaN.  A thread takes 8 columns.
template <class T>
__global__ void __launch_bounds__(256) k_q4_quantize(const T* w, int64_t ldw, int64_t V, int D, int G, uint8_t* packed, int64_t pitch,
                                                     __nv_bfloat16* scales, int groups) {
    const int tg = G / 8, per_row = groups * tg;  // threads per group (4, 8 or 16) and per row
    const int64_t total = V * per_row, padded = (total + 31) / 32 * 32;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < padded; i += (int64_t)gridDim.x * 256) {
        const bool live = i < total;
        const int64_t v = live ? i / per_row : 0;
        const int c = live ? (int)(i - v * per_row) : 0, d0 = c * 8;
        float x[8];
        uint32_t most = 0;  // bits of the largest magnitude; infinities and NaN are above all others
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = live && d0 + j < D ? to_f32(w[v * ldw + d0 + j]) : 0.f;
            most = max(most, __float_as_uint(x[j]) & 0x7FFFFFFFu);
        }
        for (int o = tg / 2; o; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        const float m = __uint_as_float(most);
        const __nv_bfloat16 sb = __float2bfloat16_rn(m / 7.f);
        const float s = __bfloat162float(sb);
        uint32_t q = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // an infinite scale: its infinities are 1 and -1 of it
            const float r = s == INFINITY ? (fabsf(x[j]) == INFINITY ? copysignf(1.f, x[j]) : 0.f)
                                          : (s > 0.f ? fminf(fmaxf(rintf(x[j] / s), -8.f), 7.f) : 0.f);
            q |= (uint32_t)((int)r + 8) << (4 * j);
        }
        if (!live) continue;
        if ((int64_t)c * 4 < pitch) *reinterpret_cast<uint32_t*>(packed + v * pitch + c * 4) = q;
        if (c % tg == 0) scales[v * groups + c / tg] = sb;
    }
}

namespace {

struct Q4Shape {
    int groups;
    int64_t pitch;
};

tt_status q4_shape(int64_t V, int32_t D, int32_t G, int32_t dtype, Q4Shape* s) {
    if (dtype != TT_F32 && dtype != TT_BF16 && dtype != TT_F16) return TT_ERR_ARG;
    if (G != 32 && G != 64 && G != 128) return TT_ERR_SHAPE;
    if (V < 1 || V > TT_HEAD_MAX_VOCAB || D < 1 || D > TT_HEAD_MAX_DIM) return TT_ERR_SHAPE;
    s->groups = (D + G - 1) / G;
    s->pitch = (int64_t)(D + 31) / 32 * 16;
    return TT_OK;
}

template <class T, int G, int NT>
struct Q4Tag {};

template <class T>
constexpr int q4_pieces() { return sizeof(T) == 4 ? 2 : 1; }

template <class T, int G, int NT>
tt_status q4_launch(Q4Args a, int sms, int dev, cudaStream_t st) {
    const int ng = a.g1 - a.g0;
    const size_t smem = (size_t)ng * (G / 32) * q4_pieces<T>() * NT * 512;
    const int64_t ntiles = (a.V + kQ4Rows - 1) / kQ4Rows;
    // warps that share a tile's columns: more of them while the tiles alone would give
    // a warp slot fewer than 4, as long as each keeps two groups
    a.ksplit = 1;
    while (a.ksplit < kQ4Warps && ntiles * a.ksplit < 4ll * sms * 2 * kQ4Warps && ng >= 4 * a.ksplit) a.ksplit *= 2;
    const int64_t per = kQ4Warps / a.ksplit, rounds = (ntiles + per - 1) / per;
    auto k = k_q4_matvec<T, G, NT>;
    if (!allow_smem<Q4Tag<T, G, NT>>(k, dev, kQ4SmemBytes)) return TT_ERR_CUDA;
    k<<<(unsigned)(rounds < 2 * sms ? rounds : 2 * sms), kQ4Threads, smem, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

template <class T, int G>
tt_status q4_rows(Q4Args a, int M, int sms, int dev, cudaStream_t st) {
    const int groups = a.groups;
    for (int m0 = 0; m0 < M; m0 += 32) {
        a.m0 = m0;
        a.M = M - m0 < 32 ? M - m0 : 32;
        const int nt = a.M <= 8 ? 1 : (a.M <= 16 ? 2 : 4);
        // x of as many groups as fit in shared memory at a time
        int fit = (int)(kQ4SmemBytes / ((size_t)(G / 32) * q4_pieces<T>() * nt * 512));
        const int launches = (groups + fit - 1) / fit;
        for (int i = 0; i < launches; ++i) {
            a.g0 = (int)((int64_t)groups * i / launches);
            a.g1 = (int)((int64_t)groups * (i + 1) / launches);
            a.accumulate = i > 0;
            const tt_status s = nt == 1 ? q4_launch<T, G, 1>(a, sms, dev, st) : (nt == 2 ? q4_launch<T, G, 2>(a, sms, dev, st) : q4_launch<T, G, 4>(a, sms, dev, st));
            if (s != TT_OK) return s;
        }
    }
    return TT_OK;
}

template <class T>
tt_status q4_type(const Q4Args& a, int M, int G, int sms, int dev, cudaStream_t st) {
    if (G == 32) return q4_rows<T, 32>(a, M, sms, dev, st);
    if (G == 64) return q4_rows<T, 64>(a, M, sms, dev, st);
    return q4_rows<T, 128>(a, M, sms, dev, st);
}

}  // namespace
}  // namespace ttemb

using namespace ttemb;

extern "C" {

tt_status tt_emb_q4_quantize(const void* weight_dev, int64_t weight_stride, int64_t vocab, int32_t dim, int32_t dtype, int32_t group,
                             uint8_t* packed_dev, uint16_t* scales_dev, tt_stream stream) {
    Q4Shape s;
    const tt_status st = q4_shape(vocab, dim, group, dtype, &s);
    if (st != TT_OK) return st;
    if (weight_stride < dim) return TT_ERR_SHAPE;
    if (!weight_dev || !packed_dev || !scales_dev || (uintptr_t)packed_dev % 16 || (uintptr_t)scales_dev % 2) return TT_ERR_ARG;
    if ((uintptr_t)weight_dev % (dtype == TT_F32 ? 4 : 2)) return TT_ERR_ARG;
    int dev = 0;
    const int sms = head_sms(&dev);
    if (sms <= 0) return TT_ERR_CUDA;
    const int64_t total = vocab * s.groups * (group / 8);
    int64_t blocks = (total + 255) / 256;
    if (blocks > 32ll * sms) blocks = 32ll * sms;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    __nv_bfloat16* sc = reinterpret_cast<__nv_bfloat16*>(scales_dev);
    if (dtype == TT_F32)
        k_q4_quantize<float><<<(unsigned)blocks, 256, 0, cs>>>(static_cast<const float*>(weight_dev), weight_stride, vocab, dim, group,
                                                               packed_dev, s.pitch, sc, s.groups);
    else if (dtype == TT_BF16)
        k_q4_quantize<__nv_bfloat16><<<(unsigned)blocks, 256, 0, cs>>>(static_cast<const __nv_bfloat16*>(weight_dev), weight_stride, vocab,
                                                                       dim, group, packed_dev, s.pitch, sc, s.groups);
    else
        k_q4_quantize<__half><<<(unsigned)blocks, 256, 0, cs>>>(static_cast<const __half*>(weight_dev), weight_stride, vocab, dim, group,
                                                                packed_dev, s.pitch, sc, s.groups);
    return cudaGetLastError() == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

tt_status tt_emb_q4_matvec(const void* x_dev, int64_t x_stride, int32_t rows, int32_t dtype, const uint8_t* packed_dev,
                           const uint16_t* scales_dev, int64_t vocab, int32_t dim, int32_t group, float* out_dev, tt_stream stream) {
    Q4Shape s;
    const tt_status st = q4_shape(vocab, dim, group, dtype, &s);
    if (st != TT_OK) return st;
    if (rows < 0 || rows > TT_Q4_MAX_ROWS || x_stride < dim) return TT_ERR_SHAPE;
    if (rows == 0) return TT_OK;
    if (!x_dev || !packed_dev || !scales_dev || !out_dev || (uintptr_t)packed_dev % 16 || (uintptr_t)scales_dev % 2 || (uintptr_t)out_dev % 4)
        return TT_ERR_ARG;
    if ((uintptr_t)x_dev % (dtype == TT_F32 ? 4 : 2)) return TT_ERR_ARG;
    int dev = 0;
    const int sms = head_sms(&dev);
    if (sms <= 0) return TT_ERR_CUDA;
    Q4Args a{};
    a.x = x_dev;
    a.ldx = x_stride;
    a.vec = (uintptr_t)x_dev % 16 == 0 && x_stride * (dtype == TT_F32 ? 4 : 2) % 16 == 0;
    a.thousand = 0x64006400u;
    a.D = dim;
    a.packed = packed_dev;
    a.pitch = s.pitch;
    a.scales = reinterpret_cast<const __nv_bfloat16*>(scales_dev);
    a.groups = s.groups;
    a.V = vocab;
    a.out = out_dev;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == TT_F32) return q4_type<float>(a, rows, group, sms, dev, cs);
    if (dtype == TT_BF16) return q4_type<__nv_bfloat16>(a, rows, group, sms, dev, cs);
    return q4_type<__half>(a, rows, group, sms, dev, cs);
}

}  // extern "C"
