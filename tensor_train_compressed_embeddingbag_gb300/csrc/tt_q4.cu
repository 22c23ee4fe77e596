// tt_q4.cu -- scores of a few rows against a table held in 4 bits (serving):
//
//   out[m, v] = sum_j scale[v, j] sum_{d in group j} (code[v, d] - 8) x[m, d]
//
// Codes are 4-bit, two to a byte (the even column in the low half), rows padded to a
// multiple of 32 columns; one bf16 scale per group of 32, 64 or 128 columns.
//
// A call reads half a byte per weight and multiplies it by the few rows of x, so
// reading the table bounds it.  What the kernel does per weight has to fit beside the
// loads: codes become 16-bit floats two at a time (an OR puts a code into the low
// mantissa bits of 128 (bf16) or 1024 (f16), one packed subtraction leaves code - 8,
// exactly), and the products run on the warp-level tensor cores
// (mma.sync.m16n8k16: 16 table rows x 8 rows of x), fp32 accumulation per group, one
// fp32 multiply-add by the group's scale into the running sum.  bf16 and f16 x enter
// as they are; an fp32 x as three bf16 pieces (8 + 8 + 8 bits of its significand), one
// MMA each: every product is exact.  The order of k inside a group is free as long as
// both operands use the same, so a thread's share of a group is one contiguous load of
// group / 8 bytes per table row, and x is laid out in shared memory in the order in
// which the fragments want it.
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
};

// (code - 8) of four columns as two 16-bit pairs: nibbles i and i + 4 of w.
template <bool BF>
__device__ __forceinline__ uint32_t q4_pair(uint32_t w, int i) {
    const uint32_t c = ((w >> (4 * i)) & 0x000F000Fu) | (BF ? 0x43004300u : 0x64006400u);
    uint32_t r;
    if (BF)
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(c), "r"(0x43084308u));  // 136
    else
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(c), "r"(0x64086408u));  // 1032
    return r;
}

template <bool BF>
__device__ __forceinline__ void mma16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <class T>
struct Q4Type {
    static constexpr bool bf = true;
    static constexpr int pieces = 1;
};
template <>
struct Q4Type<__half> {
    static constexpr bool bf = false;
    static constexpr int pieces = 1;
};
template <>
struct Q4Type<float> {
    static constexpr bool bf = true;
    static constexpr int pieces = 3;
};

// W = G / 32 words of 8 codes per thread, table row and group.  Shared memory:
// x as [group][word][piece][n tile][32 lanes] x 16 bytes: lane (g, t) of an MMA (g =
// lane / 4 the row of x, t = lane % 4) finds there x of the 8 columns that thread t
// holds in that word, in the order 0 4 1 5 2 6 3 7 of its nibbles.
template <class T, int G, int NT>
__global__ void __launch_bounds__(kQ4Threads, 2) k_q4_matvec(const __grid_constant__ Q4Args a) {
    constexpr int W = G / 32, P = Q4Type<T>::pieces;
    constexpr bool BF = Q4Type<T>::bf;
    extern __shared__ uint4 xs[];
    __shared__ float red[kQ4Warps][kQ4Rows * 8];  // one n tile at a time
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int ng = a.g1 - a.g0;

    const T* x = static_cast<const T*>(a.x);
    for (int i = threadIdx.x; i < ng * W * NT * 32; i += kQ4Threads) {
        const int l = i & 31, rest = i >> 5;
        const int nt = rest % NT, w = rest / NT % W, j = rest / NT / W;
        const int m = nt * 8 + (l >> 2), d0 = (a.g0 + j) * G + (l & 3) * (G / 4) + w * 8;
        uint16_t u[P][8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int d = d0 + (e >> 1) + (e & 1) * 4;
            const bool in = m < a.M && d < a.D;
            if (P == 1) {
                u[0][e] = in ? reinterpret_cast<const uint16_t*>(x + (a.m0 + m) * a.ldx)[d] : (uint16_t)0;
            } else {
                float v = in ? to_f32(x[(a.m0 + m) * a.ldx + d]) : 0.f;
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    const __nv_bfloat16 b = __float2bfloat16_rn(v);
                    u[p][e] = __bfloat16_as_ushort(b);
                    v -= __bfloat162float(b);
                }
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
    for (int64_t rd = blockIdx.x; rd < rounds; rd += gridDim.x) {
        const int64_t tile = rd * tiles_per_block + sub;
        float tot[2][NT][4];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) tot[r][n][e] = 0.f;
        if (tile < ntiles) {
            // four table rows per thread: tile * 32 + {0, 8, 16, 24} + g; rows past V read row V - 1
            const uint8_t* pr[4];
            const __nv_bfloat16* sr[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                int64_t v = tile * kQ4Rows + r * 8 + g;
                v = v < a.V ? v : a.V - 1;
                pr[r] = a.packed + v * a.pitch + t * (G / 8);
                sr[r] = a.scales + v * a.groups;
            }
            auto load = [&](int j, uint32_t (&q)[4][W], float (&s)[4]) {
                const int64_t at = (int64_t)(a.g0 + j) * (G / 2);
                const bool in = at + t * (G / 8) < a.pitch;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    if (W == 4) {
                        const uint4 u = in ? __ldcs(reinterpret_cast<const uint4*>(pr[r] + at))
                                           : make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
                        q[r][0] = u.x;
                        q[r][1 % W] = u.y;
                        q[r][2 % W] = u.z;
                        q[r][3 % W] = u.w;
                    } else if (W == 2) {
                        const uint2 u = in ? __ldcs(reinterpret_cast<const uint2*>(pr[r] + at)) : make_uint2(0x88888888u, 0x88888888u);
                        q[r][0] = u.x;
                        q[r][1 % W] = u.y;
                    } else {
                        q[r][0] = in ? __ldcs(reinterpret_cast<const uint32_t*>(pr[r] + at)) : 0x88888888u;
                    }
                    s[r] = __bfloat162float(sr[r][a.g0 + j]);
                }
            };
            constexpr int U = W == 4 ? 2 : 4;  // groups in flight
            uint32_t q[U][4][W];
            float s[U][4];
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (jb + i < je) load(jb + i, q[i], s[i]);
            for (int j0 = jb; j0 < je; j0 += U) {
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const int j = j0 + i;
                    if (j >= je) break;
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
                        for (int r = 0; r < 4; ++r)
#pragma unroll
                            for (int e = 0; e < 4; ++e) f[r][e] = q4_pair<BF>(q[i][r][w], e);
#pragma unroll
                        for (int p = 0; p < P; ++p)
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                const uint4 b = xs[(((j * W + w) * P + p) * NT + n) * 32 + lane];
#pragma unroll
                                for (int r = 0; r < 2; ++r) {
                                    mma16816<BF>(acc[r][n], f[2 * r][0], f[2 * r + 1][0], f[2 * r][1], f[2 * r + 1][1], b.x, b.y);
                                    mma16816<BF>(acc[r][n], f[2 * r][2], f[2 * r + 1][2], f[2 * r][3], f[2 * r + 1][3], b.z, b.w);
                                }
                            }
                    }
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                tot[r][n][e] = fmaf(s[i][2 * r + (e >> 1)], acc[r][n][e], tot[r][n][e]);
                    if (j + U < je) load(j + U, q[i], s[i]);
                }
            }
        }
        // join the warps that share the tile and write: element (row, m) of an n tile
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (n * 8 >= a.M) break;
            if (a.ksplit > 1) __syncthreads();
            float* my = red[warp];
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) my[(2 * t + (e & 1)) * kQ4Rows + r * 16 + (e >> 1) * 8 + g] = tot[r][n][e];
            if (a.ksplit > 1)
                __syncthreads();
            else
                __syncwarp();
            const int64_t v = tile * kQ4Rows + lane;
            for (int m = ks; m < 8; m += a.ksplit) {
                if (n * 8 + m >= a.M || v >= a.V) continue;
                float sum = 0.f;
                for (int k = 0; k < a.ksplit; ++k) sum += red[sub * a.ksplit + k][m * kQ4Rows + lane];
                float* o = a.out + (int64_t)(a.m0 + n * 8 + m) * a.V + v;
                *o = a.accumulate ? *o + sum : sum;
            }
            if (a.ksplit == 1) __syncwarp();
        }
    }
}

// Codes and scales of a table: per group, scale = bf16(max |w| / 7), code = w / scale
// rounded to nearest (ties to even), held within [-8, 7], plus 8.  A thread takes 8 columns.
template <class T>
__global__ void __launch_bounds__(256) k_q4_quantize(const T* w, int64_t ldw, int64_t V, int D, int G, uint8_t* packed, int64_t pitch,
                                                     __nv_bfloat16* scales, int groups) {
    const int tg = G / 8, per_row = groups * tg;  // threads per group (4, 8 or 16) and per row
    const int64_t total = V * per_row, padded = (total + 31) / 32 * 32;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < padded; i += (int64_t)gridDim.x * 256) {
        const bool live = i < total;
        const int64_t v = live ? i / per_row : 0;
        const int c = live ? (int)(i - v * per_row) : 0, d0 = c * 8;
        float x[8], m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = live && d0 + j < D ? to_f32(w[v * ldw + d0 + j]) : 0.f;
            m = fmaxf(m, fabsf(x[j]));
        }
        for (int o = tg / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const __nv_bfloat16 sb = __float2bfloat16_rn(m / 7.f);
        const float s = __bfloat162float(sb);
        uint32_t q = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float r = s > 0.f ? fminf(fmaxf(rintf(x[j] / s), -8.f), 7.f) : 0.f;
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

template <class T, int G, int NT>
tt_status q4_launch(Q4Args a, int sms, int dev, cudaStream_t st) {
    const int ng = a.g1 - a.g0;
    const size_t smem = (size_t)ng * (G / 32) * Q4Type<T>::pieces * NT * 512;
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
        int fit = (int)(kQ4SmemBytes / ((size_t)(G / 32) * Q4Type<T>::pieces * nt * 512));
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
