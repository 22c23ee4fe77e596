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
// The table stays in 8 bits until it is on the chip: TMA brings 128 rows x 128 columns of codes, four
// warps turn them into f16 (one byte permutation puts a code, made unsigned, into the mantissa of 1024; one
// packed subtraction leaves it) and write them to tensor memory, from where the MMA takes its A
// operand.  The codes of x, few against the table's, are f16 in memory from the start and come by TMA as
// the B operand.  So the accumulator's rows are table rows and its columns rows of x, and a
// warp that stores 32 lanes of a column writes 128 consecutive bytes of a row of scores.
#include <algorithm>
#include <type_traits>

#include "tt_head.cuh"

namespace ttemb {

constexpr int kQ8Threads = 512;   // warp 0: TMA, 1: MMA, 2: tensor memory, 4..7: codes to f16, 8..15: scores out
constexpr int kQ8K = 128;         // columns of a stage
constexpr int kQ8Range = 1024;    // columns that an accumulator takes (a multiple of kQ8K)
constexpr int kQ8ACols = kQ8K / 2;  // tensor-memory columns of a stage's codes

template <int BN>
struct Q8Shape {
    static constexpr uint32_t kA = 128 * kQ8K, kB = BN * kQ8K * 2, kStage = kA + kB;
    static constexpr int kStages = (BN <= 32 ? 208 : 200) * 1024 / kStage;
    static constexpr size_t kSmem = (size_t)kStages * kStage + 1024;
    static constexpr int kAcc = BN < 32 ? 32 : BN;  // columns from one accumulator to the next
    static constexpr int kAStages = 2;
    static constexpr int kACol = 2 * kAcc;
    static_assert(kACol + kAStages * kQ8ACols <= 512 && kSmem + 2048 <= 227 * 1024, "tensor and shared memory");
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

// A unit is 128 table rows x BN rows of x; the tiles of x go fastest, so blocks that run together
// share table rows.
template <int BN>
__global__ void __launch_bounds__(kQ8Threads, 1)
    k_q8_scores(const __grid_constant__ CUtensorMap map_codes, const __grid_constant__ CUtensorMap map_x, const __grid_constant__ Q8Args a) {
    using S = Q8Shape<BN>;
    constexpr int kHalf = BN / 2;        // columns of an epilogue warp
    constexpr int kRangeChunks = kQ8Range / kQ8K;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t full[S::kStages], empty[S::kStages], turned[S::kAStages], used[S::kAStages], accfull[2], accempty[2], drain;
    __shared__ uint32_t tmem_slot;
    __shared__ int gave_up_s;
    volatile int* gave_up = &gave_up_s;
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const bool lead = lane == 0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);   // the stage's MMAs are done (its codes were read before they began)
        }
        for (int i = 0; i < S::kAStages; ++i) {
            mbar_init(&turned[i], 4);  // codes are in tensor memory
            mbar_init(&used[i], 1);    // the MMAs that read them are done
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&accfull[i], 1);
            mbar_init(&accempty[i], 8);
        }
        mbar_init(&drain, 1);
        gave_up_s = 0;
    }
    if (warp == 2) tc_alloc(&tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    uint32_t it = 0;   // stages fed, turned or multiplied
    uint32_t acc = 0;  // accumulators filled or read
    bool ok = true;

    if (warp == 0) {
        for (int64_t u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
            const int v = (int)(u / a.mtiles), m = (int)(u - (int64_t)v * a.mtiles);
            for (int c = 0; c < a.chunks; ++c, ++it) {
                const uint32_t st = it % S::kStages;
                ok = head_wait(&empty[st], ((it / S::kStages) & 1) ^ 1, a.wait_ns, gave_up);
                if (!ok) break;
                if (lead) {
                    const uint32_t sa = base + st * S::kStage;
                    bulk_expect(&full[st], S::kStage);
                    tma_load2(sa, &map_codes, c * kQ8K, v * 128, &full[st]);
                    tma_load2(sa + S::kA, &map_x, c * kQ8K, m * BN, &full[st]);
                    tma_load2(sa + S::kA + S::kB / 2, &map_x, c * kQ8K + 64, m * BN, &full[st]);
                }
                __syncwarp();
            }
        }
    } else if (warp == 1) {
        const uint32_t idesc = idesc_f16(128, BN, 0, false, false);
        const uint32_t db0 = desc_lo(base + S::kA, kNoLbo);
        for (int64_t u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
            for (int r0 = 0; ok && r0 < a.chunks; r0 += kRangeChunks, ++acc) {
                const uint32_t buf = acc & 1, d = tmem + buf * S::kAcc;
                ok = head_wait(&accempty[buf], ((acc >> 1) & 1) ^ 1, a.wait_ns, gave_up);
                if (!ok) break;
                tc_fence_after();
                const int steps = min(kRangeChunks, a.chunks - r0);
                for (int c = 0; c < steps; ++c, ++it) {
                    const uint32_t st = it % S::kStages, ta = it % S::kAStages;
                    ok = head_wait(&turned[ta], (it / S::kAStages) & 1, a.wait_ns, gave_up) &&
                         head_wait(&full[st], (it / S::kStages) & 1, a.wait_ns, gave_up);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t pa = tmem + S::kACol + ta * kQ8ACols, db = db0 + st * (S::kStage >> 4);
#pragma unroll
                    for (int k = 0; k < kQ8K / 16; ++k)
                        mma_f16_ta(d, pa + k * 8, db + (k >= 4 ? (S::kB / 2) >> 4 : 0) + (k & 3) * (32 >> 4), idesc, c > 0 || k > 0, lead);
                    mma_commit(&empty[st], lead);
                    mma_commit(&used[ta], lead);
                }
                if (ok) mma_commit(&accfull[buf], lead);
            }
        }
    } else if (warp >= 4 && warp < 8) {
        const int r = (warp - 4) * 32 + lane;
        for (int64_t u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
            for (int c = 0; c < a.chunks; ++c, ++it) {
                const uint32_t st = it % S::kStages, ta = it % S::kAStages;
                ok = head_wait(&full[st], (it / S::kStages) & 1, a.wait_ns, gave_up) &&
                     head_wait(&used[ta], ((it / S::kAStages) & 1) ^ 1, a.wait_ns, gave_up);
                if (!ok) break;
                tc_fence_after();
                const uint32_t row = base + st * S::kStage + r * 128;
                const uint32_t to = tmem + ((uint32_t)((warp - 4) * 32) << 16) + S::kACol + ta * kQ8ACols;
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t q[16];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint4 w = lds16(row + (((h * 2 + x) ^ (r & 7)) << 4));  // 128-byte swizzle
                        codes_to_f16(w.x, q[x * 8], q[x * 8 + 1]);
                        codes_to_f16(w.y, q[x * 8 + 2], q[x * 8 + 3]);
                        codes_to_f16(w.z, q[x * 8 + 4], q[x * 8 + 5]);
                        codes_to_f16(w.w, q[x * 8 + 6], q[x * 8 + 7]);
                    }
                    tm_st16(to + h * 16, q);
                }
                tm_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lead) mbar_arrive(&turned[ta]);
            }
        }
    } else if (warp >= 8) {
        const int half = (warp - 8) >> 2, quad = warp & 3;
        for (int64_t u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
            const int vt = (int)(u / a.mtiles), mt = (int)(u - (int64_t)vt * a.mtiles);
            const int64_t v = (int64_t)vt * 128 + quad * 32 + lane, m0 = (int64_t)mt * BN + half * kHalf;
            int sum[kHalf];
            for (int r0 = 0; ok && r0 < a.chunks; r0 += kRangeChunks, ++acc) {
                const uint32_t buf = acc & 1;
                ok = head_wait(&accfull[buf], (acc >> 1) & 1, a.wait_ns, gave_up);
                if (!ok) break;
                tc_fence_after();
                const uint32_t t0 = tmem + buf * S::kAcc + ((uint32_t)(quad * 32) << 16) + half * kHalf;
#pragma unroll
                for (int h = 0; h < kHalf; h += 8) {
                    float x[8];
                    tm_read8(t0 + h, x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int y = __float2int_rn(x[j]);
                        sum[h + j] = r0 == 0 ? y : sum[h + j] + y;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lead) mbar_arrive(&accempty[buf]);
            }
            if (!ok) break;
            if (v < a.V && m0 < a.M) {
                const float s = a.scale[v];
                float* o = a.out + m0 * a.V + v;
                const int rows = (int)min((int64_t)kHalf, a.M - m0);
#pragma unroll
                for (int j = 0; j < kHalf; ++j) {
                    if (j < rows) *o = (float)sum[j] * (__ldg(a.xscale + m0 + j) * s);
                    o += a.V;
                }
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
            for (uint32_t i = it > S::kStages ? it - S::kStages : 0; i < it; ++i) head_drain(&full[i % S::kStages], (i / S::kStages) & 1);
        if (threadIdx.x == 32) {
            mma_commit(&drain, true);
            head_drain(&drain, 0);
        }
        __syncwarp();
        __syncthreads();
    }
    tc_fence_after();
    if (warp == 2) tc_dealloc(tmem, 512);
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

// Codes of the rows of a matrix: int8 (out8) or as f16 values (out16), columns up to `pitch` with 0.
// `lanes` threads to a row.
template <class T>
__global__ void __launch_bounds__(256) k_q8_rows(const T* x, int64_t ld, int64_t rows, int D, int lanes, int8_t* out8, __half* out16, int64_t pitch,
                                                 float* scales) {
    __shared__ uint32_t top_s[8];
    const int per = 256 / lanes, sub = threadIdx.x / lanes, lane = threadIdx.x & (lanes - 1);
    const int64_t blocks = (rows + per - 1) / per;
    for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        const int64_t r = b * per + sub;
        const bool live = r < rows;
        const T* p = x + (live ? r : 0) * ld;
        uint32_t most = 0;  // bits of the largest magnitude; infinities and NaN are above all others
        if (live)
#pragma unroll 8
            for (int d = lane; d < D; d += lanes) most = max(most, __float_as_uint(to_f32(p[d])) & 0x7FFFFFFFu);
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
        const float inv = 127.f / top;
        const bool plain = most > 0 && most < 0x7F800000u && inv < 3e38f;
#pragma unroll 4
        for (int d = lane; d < pitch; d += lanes) {
            float k = 0.f;
            if (d < D) {
                const float y = to_f32(p[d]);
                if (plain)
                    k = code_of(y, top, inv);
                else if (most == 0x7F800000u)
                    k = fabsf(y) == INFINITY ? copysignf(1.f, y) : 0.f;
                else if (most > 0 && most < 0x7F800000u)  // below 2^-120: 127 / top is infinite
                    k = code_of(y * 0x1p100f, top * 0x1p100f, 127.f / (top * 0x1p100f));
            }
            if (out8)
                out8[r * pitch + d] = (int8_t)(int)k;
            else
                out16[r * pitch + d] = __float2half_rn(k);
        }
    }
}

namespace {

bool aligned(const void* p, int to) { return (uintptr_t)p % to == 0; }

tt_status q8_sizes(int64_t rows, int64_t dim, int dtype) {
    if (dtype != TT_F32 && dtype != TT_BF16 && dtype != TT_F16) return TT_ERR_ARG;
    if (rows < 0 || rows > TT_HEAD_MAX_VOCAB || dim < 1 || dim > TT_HEAD_MAX_DIM) return TT_ERR_SHAPE;
    return TT_OK;
}

int64_t x_pitch(int64_t dim) { return (dim + 7) / 8 * 8; }
int64_t code_pitch(int64_t dim) { return (dim + 15) / 16 * 16; }

struct Q8Space {
    __half* x;
    float* xscale;
    size_t bytes;
};
Q8Space q8_space(int64_t rows, int64_t dim, void* ws) {
    const size_t codes = ((size_t)rows * x_pitch(dim) * 2 + 255) / 256 * 256;
    uint8_t* p = static_cast<uint8_t*>(ws);
    return {reinterpret_cast<__half*>(p), reinterpret_cast<float*>(p ? p + codes : nullptr), codes + ((size_t)rows * 4 + 255) / 256 * 256};
}

template <class T>
void rows_launch(const void* x, int64_t ld, int64_t rows, int D, int8_t* out8, __half* out16, int64_t pitch, float* scales, int sms, cudaStream_t st) {
    // a row's threads: so many that each has some 8 elements
    int lanes = 8;
    while (lanes < 256 && lanes * 8 < D) lanes *= 2;
    const int64_t blocks = (rows * lanes + 255) / 256;
    k_q8_rows<T><<<(unsigned)std::min<int64_t>(blocks, 16ll * sms), 256, 0, st>>>(static_cast<const T*>(x), ld, rows, D, lanes, out8, out16, pitch, scales);
}

void quantize_rows(const void* x, int64_t ld, int64_t rows, int D, int dtype, int8_t* out8, __half* out16, int64_t pitch, float* scales, int sms,
                   cudaStream_t st) {
    if (dtype == TT_F32)
        rows_launch<float>(x, ld, rows, D, out8, out16, pitch, scales, sms, st);
    else if (dtype == TT_BF16)
        rows_launch<__nv_bfloat16>(x, ld, rows, D, out8, out16, pitch, scales, sms, st);
    else
        rows_launch<__half>(x, ld, rows, D, out8, out16, pitch, scales, sms, st);
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
    k_q8_scores<BN><<<(unsigned)std::min<int64_t>(a.units, sms), kQ8Threads, Q8Shape<BN>::kSmem, st>>>(mc, mx, a);
    return cudaGetLastError() == cudaSuccess ? TT_OK : TT_ERR_CUDA;
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
    quantize_rows(weight_dev, weight_stride, rows, dim, dtype, codes_dev, nullptr, code_pitch(dim), scales_dev, sms, reinterpret_cast<cudaStream_t>(stream));
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
    quantize_rows(x_dev, x_stride, rows, dim, dtype, nullptr, w.x, x_pitch(dim), w.xscale, sms, st);
    Q8Args a{};
    a.M = rows;
    a.V = vocab;
    a.chunks = (dim + kQ8K - 1) / kQ8K;
    a.xscale = w.xscale;
    a.scale = scales_dev;
    a.out = out_dev;
    a.wait_ns = head_wait_limit();
    a.err = err_dev;
    // the narrowest tile that holds the rows; beyond 192 the width that pads less
    if (rows <= 16) return scores_launch<16>(a, codes_dev, w.x, dim, sms, dev, st);
    if (rows <= 32) return scores_launch<32>(a, codes_dev, w.x, dim, sms, dev, st);
    if (rows <= 64) return scores_launch<64>(a, codes_dev, w.x, dim, sms, dev, st);
    if (rows <= 128) return scores_launch<128>(a, codes_dev, w.x, dim, sms, dev, st);
    return scores_launch<192>(a, codes_dev, w.x, dim, sms, dev, st);
}

}  // extern "C"
