// tt_head.cuh -- device code shared by the vocabulary-head kernels (tt_head.cu):
// TMA loads, 128-byte-swizzled tensor-core operands, bounded waits.
//
// Operand tiles are 16-bit (both bf16 or both f16) and arrive by TMA with the
// 128-byte swizzle, 64 deep along K.  A tile whose matrix is contiguous along K
// ("K-major") is rows x 128 bytes: 8-row groups 1,024 bytes apart (the stride
// byte offset), one MMA's K = 16 is 32 bytes further along the row.  A tile whose
// matrix is contiguous along its M or N index ("MN-major", read transposed by the
// MMA) is made of blocks of 64 indices x 64 K rows of 128 bytes: 8-K groups 1,024
// bytes apart (stride byte offset), blocks 8,192 bytes apart (leading byte
// offset), one MMA's K = 16 is 2,048 bytes further.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "tt_tc.cuh"

namespace ttemb {

constexpr uint64_t kHeadWaitNs = 2000000000ull;  // default bound of a device wait (2 s)

__device__ __forceinline__ bool mbar_try(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// The same without the moment's suspension that try_wait allows itself.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// A warp's wait for the phase of the given parity, for at most `ns` nanoseconds (counted
// as two SM cycles each, which is a little long) or until another role of the block gave
// up; false if the phase did not complete.  The answer is the same in every lane, and
// known to the compiler to be so: what the TMA and MMA warps compute between waits
// stays in uniform registers, where the tensor instructions take their operands from.
__device__ __forceinline__ bool head_wait(uint64_t* bar, uint32_t parity, uint64_t ns, volatile int* gave_up) {
    if (ns == 0) return __all_sync(0xffffffffu, mbar_test(bar, parity));
    if (__all_sync(0xffffffffu, mbar_try(bar, parity))) return true;
    const int64_t t0 = clock64();
    while (!__all_sync(0xffffffffu, mbar_try(bar, parity))) {
        if (__any_sync(0xffffffffu, *gave_up || (uint64_t)(clock64() - t0) >= 2 * ns)) return false;
    }
    return true;
}

// The same wait without the early way out, for copies and MMAs in flight.
__device__ __forceinline__ void head_drain(uint64_t* bar, uint32_t parity) {
    const int64_t t0 = clock64();
    while (!mbar_try(bar, parity)) {
        if ((uint64_t)(clock64() - t0) >= 2 * kHeadWaitNs) return;
    }
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// One box of a 3-D tensor map into shared memory.  x: innermost coordinate, a
// multiple of 8 elements (16 bytes).
__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

// Shared-memory matrix descriptor of a 128-byte-swizzled operand, in two words: the
// start address (moving along K or to another tile adds to it) with the leading byte
// offset (lbo: bytes between the 64-index blocks of an MN-major operand), and the rest.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | (lbo >> 4 << 16); }
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;  // stride 1,024 bytes, version, 128-byte swizzle
constexpr uint32_t kNoLbo = 16;                                   // K-major: unused, written as 1

// Instruction descriptor of kind::f16, fp32 accumulator; fmt 0: f16, 1: bf16.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int fmt, bool a_mn, bool b_mn) {
    return (1u << 4) | ((uint32_t)fmt << 7) | ((uint32_t)fmt << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// One MMA (K = 16), run by a whole warp and issued by the lane whose `lead` is set.
__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool accumulate, bool lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "mov.b64 da, {%1, %6};\n\tmov.b64 db, {%2, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"((uint32_t)accumulate), "r"((uint32_t)lead), "r"(kDescHi)
        : "memory");
}

// The same with A in tensor memory (K-major: a row per lane, two 16-bit elements per column).
__device__ __forceinline__ void mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, bool accumulate, bool lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "mov.b64 db, {%2, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"((uint32_t)accumulate), "r"((uint32_t)lead), "r"(kDescHi)
        : "memory");
}

__device__ __forceinline__ void axpy2(float& x, float& y, float ax, float ay, float f) {
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 c, {%0, %1};\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(ax), "f"(ay), "f"(f));
}

// 16 bytes from global to shared memory without a register (zeros if !have); done after
// the thread's cp_wait.  What the other lanes of a warp copied is seen after a __syncwarp.
__device__ __forceinline__ void cp16(void* dst, const void* src, bool have) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(have ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The mbarrier's phase completes when every MMA issued so far by the lead lane is done.
__device__ __forceinline__ void mma_commit(uint64_t* bar, bool lead) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar)),
        "r"((uint32_t)lead)
        : "memory");
}

// Two fp32 operations in one instruction, each rounded as the single one is.
__device__ __forceinline__ void fma2(float& x, float& y, float ax, float ay, float bx, float by) {
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\tmov.b64 c, {%4, %5};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(ax), "f"(ay), "f"(bx), "f"(by));
}
__device__ __forceinline__ void mul2(float& x, float& y, float ax, float ay) {
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\tmul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(ax), "f"(ay));
}
__device__ __forceinline__ void add2(float& x, float& y, float ax, float ay) {
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\tadd.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(ax), "f"(ay));
}

// Start reading 32 consecutive fp32 columns of this warp's 32 lanes (lane i gets its
// row); the values may be used after tm_wait_ld on the same array.
__device__ __forceinline__ void tm_ld32(uint32_t taddr, float (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]),
          "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]),
          "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]),
          "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr));
}
// All reads started so far are done.  The array passes through the statement, so
// nothing that uses it can be moved above the wait.
__device__ __forceinline__ void tm_wait_ld(float (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]),
                   "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]),
                   "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]),
                   "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
                 :
                 : "memory");
}
// The same for 16 columns, waited for at once.
__device__ __forceinline__ void tm_read16(uint32_t taddr, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]),
          "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tm_read8(uint32_t taddr, float (&v)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
        : "r"(taddr)
        : "memory");
}
// Write 16 columns of this warp's 32 lanes (32 16-bit elements of an A operand's row);
// tm_wait_st makes all such writes done.
__device__ __forceinline__ void tm_st16(uint32_t taddr, const uint32_t (&w)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "r"(w[8]), "r"(w[9]), "r"(w[10]), "r"(w[11]),
        "r"(w[12]), "r"(w[13]), "r"(w[14]), "r"(w[15])
        : "memory");
}
// One column of this warp's lanes, read (waited for) and written.
__device__ __forceinline__ uint32_t tm_read1(uint32_t taddr) {
    uint32_t v;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;" : "=r"(v) : "r"(taddr) : "memory");
    return v;
}
__device__ __forceinline__ void tm_write1(uint32_t taddr, uint32_t v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(v) : "memory");
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Running maximum and sum of exp over one more 32 scores of a row, of which the first
// `valid` count.  v is in units of which c makes log2 units (c > 0); the maximum is kept in
// log2 units, which are the same for every tile of the table whatever its scale.
__device__ __forceinline__ void take_scores(float (&v)[32], int64_t valid, float c, float& run_m, float& run_s) {
    if (valid < 32) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j >= valid) v[j] = -INFINITY;
    }
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < 32; j += 2) mx[(j >> 1) & 3] = fmaxf(fmaxf(mx[(j >> 1) & 3], v[j]), v[j + 1]);
    const float mn = fmaxf(run_m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c);
    const float m2 = mn == -INFINITY ? 0.f : mn;
    float s[4] = {run_s * ex2(run_m - m2), 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
        fma2(v[j], v[j + 1], c, c, -m2, -m2);
        fma2(v[j + 2], v[j + 3], c, c, -m2, -m2);
        add2(s[0], s[1], ex2(v[j]), ex2(v[j + 1]));
        add2(s[2], s[3], ex2(v[j + 2]), ex2(v[j + 3]));
    }
    run_s = (s[0] + s[1]) + (s[2] + s[3]);
    run_m = mn;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <class T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }

// Two floats rounded to nearest and packed, the first in the low half; fmt 0: f16, 1: bf16.
__device__ __forceinline__ uint32_t pack16(float a, float b, int fmt) {
    uint32_t r;
    if (fmt)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
// The hi pieces of two fp32 operands: infinities become the largest f16, and what is left
// of them, the lo piece, infinite.  So one product of an infinity (with the other operand's hi
// piece, which has its sign) is infinite and none is inf - inf or infinity times a lo piece of 0.
__device__ __forceinline__ uint32_t pack_hi(float a, float b) {
    uint32_t r;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
// 32 floats rounded and packed; one branch on the type.
__device__ __forceinline__ void pack32(const float (&p)[32], uint32_t (&q)[16], int fmt) {
    if (fmt) {
#pragma unroll
        for (int j = 0; j < 16; ++j) q[j] = pack16(p[2 * j], p[2 * j + 1], 1);
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) q[j] = pack16(p[2 * j], p[2 * j + 1], 0);
    }
}
__device__ __forceinline__ float2 unpack_f16(uint32_t v) { return __half22float2(*reinterpret_cast<__half2*>(&v)); }

// Exponent of the power of two that brings a tensor whose largest finite magnitude has
// these fp32 bits just below 2^14 (the largest f16 is 65,504); 0 for an all-zero one.
__device__ __forceinline__ int scale_exp(uint32_t absmax_bits) {
    if (absmax_bits == 0 || absmax_bits >= 0x7F800000u) return 0;
    return min(13 - ((int)(absmax_bits >> 23) - 127), 126);
}
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }
// The same for any e, held within fp32's normal range.
__device__ __forceinline__ float exp2c(int e) { return exp2i(max(-126, min(127, e))); }
// 2^e as a product, which undoes two scales of any size: b is 1 unless a alone falls short.
struct Pow2 {
    float a, b;
    __device__ __forceinline__ explicit Pow2(int e) : a(exp2c(e)), b(exp2c(e - max(-126, min(127, e)))) {}
    __device__ __forceinline__ float operator()(float x) const { return x * b * a; }
    __device__ __forceinline__ void operator()(float (&v)[32]) const {
        if (b != 1.f) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] *= b;
        }
        if (a != 1.f) {
#pragma unroll
            for (int j = 0; j < 32; j += 2) mul2(v[j], v[j + 1], a, a);
        }
    }
};
__device__ __forceinline__ int amax_exp(const uint32_t* p) { return p ? scale_exp(*p) : 0; }

// How the fused kernels share their work: the tiles (x, y), all y of one x before the
// next x, are cut into `blocks` equal runs.  A run's tiles of one x are a segment; an x
// whose tiles lie in one run is whole, others are joined from their runs' segments.
struct Runs {
    int xtiles, ytiles, blocks;
    __host__ __device__ int64_t total() const { return (int64_t)xtiles * ytiles; }
    __host__ __device__ int64_t begin(int b) const { return total() * b / blocks; }
    __host__ __device__ int block_of(int64_t t) const { return (int)(((t + 1) * blocks - 1) / total()); }
    __host__ __device__ int first(int64_t x) const { return block_of(x * ytiles); }
    __host__ __device__ int last(int64_t x) const { return block_of(x * ytiles + ytiles - 1); }
};

// Where a product goes: converted rows of `out`, or (out null) fp32 partial sums, one
// array per K range.
struct OutArgs {
    void* out;       // [M][ldo] of `type`
    int64_t ldo;
    int type;        // tt_dtype
    int vec;         // rows of out are 16-byte aligned
    float* partial;  // [splits][M][pp], pp a multiple of 32
    int64_t pp;
    int accumulate;  // add to what partial holds
};

__device__ __forceinline__ void store_one(void* out, int64_t at, float v, int type) {
    if (type == TT_F32)
        static_cast<float*>(out)[at] = v;
    else if (type == TT_BF16)
        static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
    else
        static_cast<__half*>(out)[at] = __float2half_rn(v);
}

// A warp's 32 rows x 64 bytes, a row per lane, written out through 2 KB of shared memory
// so that four lanes write one row's 64 bytes and a store touches 8 rows, not 32.  base:
// where the first row's bytes go; rows past `rows` are left alone.
__device__ __forceinline__ void put_rows(uint4* buf, const uint4 (&mine)[4], uint8_t* base, int64_t pitch, int64_t rows) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 4; ++c) buf[lane * 4 + (c ^ ((lane >> 1) & 3))] = mine[c];
    __syncwarp();
    const int r0 = lane >> 2, c = lane & 3;
    const uint4* from = buf + r0 * 4 + (c ^ ((r0 >> 1) & 3));  // 8 rows on, the swizzle is the same
    uint8_t* to = base + r0 * pitch + c * 16;
    if (rows >= 32) {
#pragma unroll
        for (int i = 0; i < 4; ++i, to += 8 * pitch) *reinterpret_cast<uint4*>(to) = from[i * 32];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i, to += 8 * pitch)
            if (r0 + i * 8 < rows) *reinterpret_cast<uint4*>(to) = from[i * 32];
    }
}
__device__ __forceinline__ uint4 bits4(const float* v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
// The same for 32 fp32 columns (128 bytes a row).
__device__ __forceinline__ void put_rows_f32(uint4* buf, const float (&v)[32], uint8_t* base, int64_t pitch, int64_t rows) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint4 mine[4] = {bits4(v + h * 16), bits4(v + h * 16 + 4), bits4(v + h * 16 + 8), bits4(v + h * 16 + 12)};
        put_rows(buf, mine, base + h * 64, pitch, rows);
    }
}
__device__ __forceinline__ void put_rows_16(uint4* buf, const float (&v)[32], uint8_t* base, int64_t pitch, int64_t rows, int fmt) {
    uint32_t q[16];
    pack32(v, q, fmt);
    const uint4 mine[4] = {make_uint4(q[0], q[1], q[2], q[3]), make_uint4(q[4], q[5], q[6], q[7]), make_uint4(q[8], q[9], q[10], q[11]),
                           make_uint4(q[12], q[13], q[14], q[15])};
    put_rows(buf, mine, base, pitch, rows);
}

// The same for rows that do not begin on 16-byte boundaries, and their last columns: lanes
// along a row, element by element.  cols: how many of the 32 columns there are.
__device__ __forceinline__ void put_elements(uint4* buf, const float (&v)[32], void* base, int64_t ld, int64_t rows, int64_t cols, int type) {
    const int lane = threadIdx.x & 31, nrows = (int)min(rows, (int64_t)32), ncols = (int)min(cols, (int64_t)32);
    if (type == TT_F32) {
        const int k = lane & 15, r0 = lane >> 4;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 4; ++c) buf[lane * 4 + (c ^ ((lane >> 1) & 3))] = bits4(v + h * 16 + c * 4);
            __syncwarp();
            float* to = static_cast<float*>(base) + r0 * ld + h * 16 + k;
            if (h * 16 + k < ncols) {
#pragma unroll 4
                for (int i = 0; i < 16; ++i, to += 2 * ld)
                    if (i * 2 + r0 < nrows) *to = reinterpret_cast<const float*>(buf)[(i * 2 + r0) * 16 + ((k >> 2) ^ (i & 3)) * 4 + (k & 3)];
            }
        }
    } else {
        uint32_t q[16];
        pack32(v, q, type == TT_BF16);
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 4; ++c) buf[lane * 4 + (c ^ ((lane >> 1) & 3))] = make_uint4(q[4 * c], q[4 * c + 1], q[4 * c + 2], q[4 * c + 3]);
        __syncwarp();
        uint16_t* to = static_cast<uint16_t*>(base) + lane;
        if (lane < ncols) {
#pragma unroll 8
            for (int r = 0; r < 32; ++r, to += ld)
                if (r < nrows) *to = reinterpret_cast<const uint16_t*>(buf)[r * 32 + ((lane >> 3) ^ ((r >> 1) & 3)) * 8 + (lane & 7)];
        }
    }
}

// The target elements of dz lose their low bits in 16 bits.  Over many rows these
// roundings average out; with few targets in the whole batch the gradients carry each of
// them whole (up to 2^-8 or 2^-11, where their own rounding is of that size at most), so
// what they lost is added where dhidden's fp32 sums are joined.  K = 0: not done.
struct Residue {
    const int* ids;    // [K][rows]
    const float* dzt;  // times to_own: in dhidden's units
    const float* to_own;
    const void* w;
    int64_t ldw, rows;
    int K, fmt;
    // of dhidden[n][c]
    __device__ __forceinline__ float operator()(int64_t n, int c) const {
        float s = 0.f;
        for (int k = 0; k < K; ++k) {
            const int id = ids[k * rows + n];
            bool first = id >= 0;  // the same id further on is the same element
            for (int j = 0; j < k; ++j) first &= ids[j * rows + n] != id;
            if (!first) continue;
            const float x = dzt[k * rows + n] * to_own[n];
            const uint32_t b = pack16(x, 0.f, fmt) & 0xFFFFu;
            const uint16_t y = static_cast<const uint16_t*>(w)[id * ldw + c];
            s = fmaf(x - (fmt ? __uint_as_float(b << 16) : unpack_f16(b).x), fmt ? __uint_as_float((uint32_t)y << 16) : unpack_f16(y).x, s);
        }
        return s;
    }
};

// Columns [col, col + 32), col < N, of a warp's 32 rows from row0 < M on, a row per lane.
__device__ __forceinline__ void store_out(const OutArgs& o, uint4* buf, int split, int64_t row0, int64_t col, int64_t M, int64_t N, float (&v)[32],
                                          Pow2 sc) {
    const int lane = threadIdx.x & 31;
    const int64_t rows = M - row0;
    if (o.out) {
        sc(v);
        const int64_t at = row0 * o.ldo + col;
        if (o.vec && col + 32 <= N) {
            if (o.type == TT_F32)
                put_rows_f32(buf, v, reinterpret_cast<uint8_t*>(static_cast<float*>(o.out) + at), o.ldo * 4, rows);
            else
                put_rows_16(buf, v, reinterpret_cast<uint8_t*>(static_cast<uint16_t*>(o.out) + at), o.ldo * 2, rows, o.type == TT_BF16);
        } else {
            put_elements(buf, v, static_cast<uint8_t*>(o.out) + at * (o.type == TT_F32 ? 4 : 2), o.ldo, rows, N - col, o.type);
        }
    } else {  // whole chunks: the columns past N hold zeros
        float* p = o.partial + ((int64_t)split * M + row0) * o.pp + col;
        if (o.accumulate && lane < rows) {
            const float4* y4 = reinterpret_cast<const float4*>(p + lane * o.pp);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float4 y = y4[q];
                v[4 * q] += y.x;
                v[4 * q + 1] += y.y;
                v[4 * q + 2] += y.z;
                v[4 * q + 3] += y.w;
            }
        }
        put_rows_f32(buf, v, reinterpret_cast<uint8_t*>(p), o.pp * 4, rows);
    }
}

// ---------------------------------------------------------------- host

constexpr int kMaxHeadDevices = 64;

// Multiprocessors of the current device, 0 if there is none; asked once per device.
inline int head_sms(int* device = nullptr) {
    static std::atomic<int> known[kMaxHeadDevices];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxHeadDevices) {
        cudaGetLastError();
        return 0;
    }
    if (device) *device = dev;
    n = known[dev].load(std::memory_order_relaxed);
    if (n) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    known[dev].store(n, std::memory_order_relaxed);
    return n;
}

uint64_t head_wait_limit();  // bound of each device wait, ns (tt_emb_head_set_wait_limit)

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder of tensor maps, null without one.
inline EncodeTiled encode_tiled() {
    static EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// A kernel's dynamic shared memory limit on the current device, set once per device
// (K: a tag of the kernel's own).
template <class K, class F>
bool allow_smem(F* kernel, int device, size_t bytes) {
    static std::atomic<bool> done[kMaxHeadDevices];
    if (done[device].load(std::memory_order_relaxed)) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    done[device].store(true, std::memory_order_relaxed);
    return true;
}

}  // namespace ttemb
