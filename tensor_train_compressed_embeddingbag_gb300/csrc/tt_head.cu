// tt_head.cu -- the vocabulary head: softmax cross entropy and distillation from a
// teacher's top logits over z[n, v] = <hidden[n], weight[v]>, forward and backward,
// without an N x V array of logits.
//
//   lse[n]  = log sum_v exp(z[n, v] / T)
//   xent    loss[n] = lse[n] - z[n, t_n]                                   (T = 1)
//   distill q[n, k] = softmax over the row's entries of teacher_logit / T,
//           loss[n] = T^2 sum_k q[n, k] (log q[n, k] - z[n, id_k] / T + lse[n])
//   dz[n, v] = g_n T (exp(z[n, v] / T - lse[n]) - q[n, v])    (q: one-hot for xent)
//   dhidden = dz weight,  dweight = dz^T hidden
//
// Forward: one product kernel keeps, per row, a running maximum and sum of the
// exponentials of its column tiles and writes one pair per strip of tiles; a row
// kernel joins them and takes the target scores as fp32 dot products.
// Backward, D <= 128: one kernel per gradient, each forming the scores again and
// keeping dz on the chip (tt_head_fused.cuh).  Wider: the table is taken in pieces of
// the vocabulary.  For each, the scores are formed again, dz of the piece is written
// in 16 bits (k_head_fix then writes the entries that have a target), and two products
// read it: dweight of the piece and the piece's share of dhidden.  The only array of
// N x (vocabulary piece) is that dz (at most kDzBytes, or 1,024 columns).
//
// Types.  bf16 and f16 inputs go to the tensor cores as they are.  An fp32 input x
// is split as x 2^e = hi + lo with hi, lo in f16 and a product is taken as hi hi + hi lo +
// lo hi; e is a power-of-two scale that puts the largest magnitude near 2^14: of a hidden
// row in the forward pass, of 128 x 128 elements of the table, of all hidden rows that
// count in the backward pass.  So an element enters with 22 bits, or to 2^-39 of the largest
// one under its scale where that is more; fp32 accumulation; lo lo (2^-22 of the product and
// below) is dropped.
//
// dz is rounded to the inputs' 16-bit type before the two gradient products (by at most 2^-8
// or 2^-11 of an entry, independent errors, the size of the gradients' own final rounding),
// and split like an input for fp32.  For f16 and fp32 it is scaled as well, by a power of two that
// puts |g T| just below 2^14: an element keeps its bits down to 2^-28 of |g T| (fp32's two
// pieces: 22 bits down to 2^-16, to 2^-39 absolute below).  For dhidden that is the row's own
// g (or 2^-100 of the largest, if that is more), as rows are independent of each other.  For
// dweight, a sum over rows, the batch's largest |g T| is the measure: D > 128 has one dz for
// both products, and the hidden rows that dweight multiplies it by take the factor between
// the two scales; k_head_fused, whose hidden rows form the scores as well, scales dz, and
// what lies below 2^-39 of the batch's largest |g T| is lost to dweight there.
#include <math.h>

#include <type_traits>

#include "tt_head.cuh"
#include "tt_head_few.cuh"
#include "tt_head_fused.cuh"
#include "tt_head_gemm.cuh"

namespace ttemb {

constexpr int64_t kDzBytes = 256ll << 20;  // dz of one vocabulary piece: four pieces at 4096 x 131072, where a product fills the SMs many times over
constexpr int64_t kMaxBlocks = 1ll << 26;    // 32 x 32 blocks of targets (1 GB of them)
constexpr int kFewMinDim = 256;              // 16-bit rows: k_head_few from this width on
// 16-bit types, this many targets in all: their share of the gradients in fp32.  Error of the
// gradients against their rounding alone (bf16, 2 x 90656 x 812; worst of six): 2.3 without,
// 1.0 here; with more targets it is 1.4 to 1.5 and steady.  It costs a launch of 3 to 12 us.
constexpr int kFewTargets = 64;
constexpr int kMaxTeacher = TT_HEAD_MAX_TEACHER;

// ---------------------------------------------------------------- rows and copies

struct HeadIn {
    const void* h;
    const void* w;
    int64_t ldh, ldw;  // elements between rows
    int64_t N, V;
    int D, Dp;         // Dp: D rounded up to 8, the row pitch of packed copies
    int vec;           // rows of h and w are 16-byte aligned and D is a multiple of 8
};

// What a row is trained towards.
struct Target {
    const int64_t* ids;    // [N][K]; xent: the targets, K = 1
    const float* logits;   // [N][K] teacher logits; null: xent
    int64_t ignore;        // xent: the id of rows that do not count
    int K;
    float T;
};

// Whether xent row n counts; ids that are neither `ignore` nor in [0, V) are
// recorded and do not count.
__device__ __forceinline__ int64_t xent_id(const Target& t, int64_t n, int64_t V, int* err) {
    const int64_t id = t.ids[n];
    if (id == t.ignore) return -1;
    if (id < 0 || id >= V) {
        if (err) atomicOr(err, kErrIndex);
        return -1;
    }
    return id;
}

// The dot products of x with U rows y[.], side by side: their loads are in flight together.
template <int U, class T>
__device__ __forceinline__ void warp_dots(const T* x, const T* const (&y)[U], int D, int vec, int lane, float (&out)[U]) {
    constexpr int E = 16 / sizeof(T);
    float s[U][2] = {};
    if (vec) {
#pragma unroll(U == 1 ? 4 : 2)
        for (int i = lane * E; i < D; i += 32 * E) {
            const uint4 a = *reinterpret_cast<const uint4*>(x + i);
            uint4 b[U];
#pragma unroll
            for (int u = 0; u < U; ++u) b[u] = *reinterpret_cast<const uint4*>(y[u] + i);
            const T* pa = reinterpret_cast<const T*>(&a);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const T* pb = reinterpret_cast<const T*>(&b[u]);
#pragma unroll
                for (int j = 0; j < E; ++j) s[u][j & 1] = fmaf(to_f32(pa[j]), to_f32(pb[j]), s[u][j & 1]);
            }
        }
    } else {
#pragma unroll(U == 1 ? 16 : 4)
        for (int i = lane; i < D; i += 32) {
            const float a = to_f32(x[i]);
#pragma unroll
            for (int u = 0; u < U; ++u) s[u][0] = fmaf(a, to_f32(y[u][i]), s[u][0]);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) out[u] = s[u][0] + s[u][1];
#pragma unroll
    for (int o = 16; o; o >>= 1) {
#pragma unroll
        for (int u = 0; u < U; ++u) out[u] += __shfl_xor_sync(0xffffffffu, out[u], o);
    }
}

template <class T>
__device__ __forceinline__ float warp_dot(const T* x, const T* y, int D, int vec, int lane) {
    const T* const rows[1] = {y};
    float out[1];
    warp_dots<1>(x, rows, D, vec, lane, out);
    return out[0];
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A warp's join of a row's (maximum, sum) pairs; natural-log sum in every lane.
__device__ __forceinline__ float join_parts(const float2* p, int n, int lane) {
    float m = -INFINITY, s = 0.f;
    for (int i = lane; i < n; i += 32) {
        const float2 x = p[i];
        const float mn = fmaxf(m, x.x), b = mn == -INFINITY ? 0.f : mn;
        s = s * ex2(m - b) + x.y * ex2(x.x - b);
        m = mn;
    }
    const float mn = warp_max(m), b = mn == -INFINITY ? 0.f : mn;
    s = warp_sum(s * ex2(m - b));
    return (b + log2f(s)) * kLn2;
}

__device__ __forceinline__ void split1(float x, uint16_t& hi, uint16_t& lo) {
    const uint32_t h = pack_hi(x, 0.f);
    hi = (uint16_t)h;
    lo = __half_as_ushort(__float2half_rn(x - unpack_f16(h).x));
}

constexpr int kRowThreads = 128;  // per row or four rows; wide: per row, when rows are few and have many entries
constexpr int kRowThreadsWide = 512;
constexpr int kAmaxShares = 64;  // blocks that look for the largest magnitudes

// The teacher's distribution of one row, a block per row (red: two floats per warp): q[k] and log q[k] in
// shared memory, ids as int (-1: not counted).  An id below 0 marks an entry that
// does not count, whatever its logit holds; one past the table is recorded and does
// not count either; so does an entry whose logit is -inf.  Returns whether any counts.
template <int RT>
__device__ bool teacher_row(const Target& t, int64_t n, int64_t V, float* q, float* logq, int* ids, float* red, int* err) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float mx = -INFINITY;
    for (int k = tid; k < t.K; k += RT) {
        const int64_t id = t.ids[n * t.K + k];
        float x = -INFINITY;
        int got = -1;
        if (id >= V) {
            if (err) atomicOr(err, kErrIndex);
        } else if (id >= 0) {
            x = t.logits[n * t.K + k];
            got = x == -INFINITY ? -1 : (int)id;
        }
        logq[k] = x;
        ids[k] = got;
        if (got >= 0) mx = (mx != mx || x != x) ? NAN : fmaxf(mx, x);
    }
    // a NaN logit makes the whole row NaN, as a softmax does
    const bool nan = __syncthreads_or(mx != mx);
    mx = warp_max(mx);
    if (lane == 0) red[warp] = mx;
    __syncthreads();
    for (int i = 0; i < RT / 32; ++i) mx = fmaxf(mx, red[i]);
    if (nan) mx = NAN;
    float s = 0.f;
    for (int k = tid; k < t.K; k += RT)
        if (ids[k] >= 0) s += expf((logq[k] - mx) / t.T);
    s = warp_sum(s);
    if (lane == 0) red[RT / 32 + warp] = s;
    const bool any = __syncthreads_or(mx != -INFINITY);
    s = 0.f;
    for (int i = 0; i < RT / 32; ++i) s += red[RT / 32 + i];
    const float ls = logf(s), inv = 1.f / s;
    for (int k = tid; k < t.K; k += RT) {
        const float d = (logq[k] - mx) / t.T;
        q[k] = ids[k] >= 0 ? expf(d) * inv : 0.f;
        logq[k] = ids[k] >= 0 ? d - ls : 0.f;
    }
    __syncthreads();
    return any;
}

// Scores of a row's teacher entries (but those with q = 0), four to a warp at a time, one
// where there are warps for that.  give(k, z) is called by one lane per entry.  The entries'
// rows are scattered reads, bound by how many are in flight: bf16, 2048 rows x 64 entries of
// width 1024, 268 MB, 45 us (6.0 TB/s); one entry at a time 66 to 80.
template <int RT, class T, class F>
__device__ __forceinline__ void entry_scores(const HeadIn& in, int64_t n, int K, const float* q, const int* ids, F give) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T* h = static_cast<const T*>(in.h) + n * in.ldh;
    const T* w = static_cast<const T*>(in.w);
    constexpr int U = RT == kRowThreadsWide ? 1 : 4;
    for (int k = warp * U; k < K; k += RT / 32 * U) {
        const T* rows[U];
        bool some = false;
#pragma unroll
        for (int u = 0; u < U; ++u) {  // entries that are not there read the hidden row itself
            const bool is = k + u < K && q[k + u] != 0.f;
            rows[u] = is ? w + (int64_t)ids[k + u] * in.ldw : h;
            some |= is;
        }
        if (!some) continue;
        float z[U];
        warp_dots<U>(h, rows, in.D, in.vec, lane, z);
        float mine = z[0];
#pragma unroll
        for (int u = 1; u < U; ++u) mine = lane == u ? z[u] : mine;
        if (lane < U && k + lane < K && q[k + lane] != 0.f) give(k + lane, mine);
    }
}

// lse and loss of every row: the strips' pairs joined, the target scores as dot
// products.  xent: a warp per row; distill: a block per row, a warp per entry.
template <class T, bool DISTILL, int RT>
__global__ void __launch_bounds__(RT) k_head_finish(HeadIn in, Target t, const float2* part, int slots, int per_slot, Runs runs,
                                                             float* loss, float* lse, int* err) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T* h = static_cast<const T*>(in.h);
    const T* w = static_cast<const T*>(in.w);
    const auto row_lse = [&](int64_t n) {  // of the slots, those that the row's runs filled
        const int used = runs.blocks ? runs.last(n / 128) - runs.first(n / 128) + 1 : slots;
        return join_parts(part + n * slots * per_slot, used * per_slot, lane);
    };
    if (!DISTILL) {
        const int64_t n = (int64_t)blockIdx.x * (RT / 32) + warp;
        if (n >= in.N) return;
        const int64_t id = xent_id(t, n, in.V, lane == 0 ? err : nullptr);
        const float z = id >= 0 ? warp_dot(h + n * in.ldh, w + id * in.ldw, in.D, in.vec, lane) : 0.f;
        const float l = row_lse(n);
        if (lane == 0) {
            lse[n] = l;
            loss[n] = id >= 0 ? l - z : 0.f;
        }
    } else {
        extern __shared__ float sm[];
        float* q = sm;
        float* lq = sm + t.K;
        int* ids = reinterpret_cast<int*>(sm + 2 * t.K);
        __shared__ float red[RT / 16];
        __shared__ float ls;
        const int64_t n = blockIdx.x;
        const bool any = teacher_row<RT>(t, n, in.V, q, lq, ids, red, err);
        if (warp == 0) {
            const float l = row_lse(n);
            if (lane == 0) ls = l;
        }
        __syncthreads();
        const float l = ls;
        float acc = 0.f;
        entry_scores<RT, T>(in, n, t.K, q, ids, [&](int k, float z) { acc += q[k] * (lq[k] - z / t.T + l); });
        acc = warp_sum(acc);
        __syncthreads();
        if (lane == 0) red[warp] = acc;
        __syncthreads();
        if (threadIdx.x == 0) {
            lse[n] = l;
            float sum = 0.f;
            for (int i = 0; i < RT / 32; ++i) sum += red[i];
            loss[n] = any ? t.T * t.T * sum : 0.f;
        }
    }
}

// What the backward pass needs of every row, a block per row: its weight (g T, 0 for a
// row that does not count) under its own scale and under the batch's, its lse in log2
// units, dz of its target entries under the batch's, and its packed copy.  A row that does
// not count, and what fills up a tile of k_head_fused, is all ones with an lse that makes every
// p 0: nothing that it holds, infinities and NaN included, reaches dweight, and a table row
// that is scored -inf by a column of its own is so there too (zeros would make it NaN).
// Entries of one row with the same id hold the same value, of their summed q.  Target
// entries go to arrays [K][N] (ids, dzt) and, for k_head_fused, to their 32 x 32 blocks.
struct RowsArgs {
    const float* lse;
    const float* grad;
    const uint32_t* shares;  // fp32, f16: the largest magnitudes, joined in
    uint32_t* amax;          //   [0] hidden's, [2] |g T|'s; null: no scales
    int* zexp;               //   exponent of the row's own scale over the batch's
    float *nlse, *scale, *scale_batch;  // the last may be scale
    float* to_own;  // from the batch's scale to the row's
    int* ids;
    float* dzt;
    TargetBlock* blocks;
    int nblocks;
    TargetEntry* ents;
    uint16_t* hp;
    int64_t hrows;  // rows of hp
    uint16_t* hq;  // null, or hidden rows under hidden's scale, less what the row's has over the batch's, for dweight
    uint16_t one;  // 1 in hp's type
    int* err;
};
constexpr float kNoLse = -3e38f;  // -lse of a row that does not count
template <class T, bool DISTILL, int RT>
__global__ void __launch_bounds__(RT)
    k_head_rows(HeadIn in, Target t, const __grid_constant__ RowsArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t n = blockIdx.x;
    const T* h = static_cast<const T*>(in.h) + n * in.ldh;
    const T* w = static_cast<const T*>(in.w);
    if (n >= in.N) {
        if (threadIdx.x == 0) {
            a.nlse[n] = kNoLse;
            a.scale[n] = a.scale_batch[n] = a.to_own[n] = 0.f;
        }
        for (int i = threadIdx.x; i < in.Dp; i += RT) {
            a.hp[n * in.Dp + i] = a.one;
            if (sizeof(T) == 4) a.hp[(a.hrows + n) * in.Dp + i] = 0;
        }
        return;
    }
    const float l = a.lse[n];
    bool any;
    extern __shared__ float sm[];
    __shared__ float red[RT / 16];
    float* q = sm;
    int* ids = reinterpret_cast<int*>(sm + 2 * t.K);
    int64_t xid = -1;
    if (DISTILL) {
        any = teacher_row<RT>(t, n, in.V, q, sm + t.K, ids, red, a.err);
    } else {
        xid = xent_id(t, n, in.V, threadIdx.x == 0 ? a.err : nullptr);
        any = xid >= 0;
    }
    const float gt = any ? a.grad[n] * t.T : 0.f;
    int ez = 0, eh = 0, own = 0;  // own: the row's scale over the batch's
    if (a.amax) {  // the shares of the largest magnitudes joined: dz's by warps 0 and 1, hidden's by 2 and 3
        __shared__ uint32_t most[4];
        static_assert(kRowThreads == 2 * kAmaxShares, "a share per thread of the first four warps");
        if (warp < 4) {
            const uint32_t m = __reduce_max_sync(0xffffffffu, a.shares[threadIdx.x]);
            if (lane == 0) most[warp] = m;
        }
        __syncthreads();
        const uint32_t mz = max(most[0], most[1]), mh = max(most[2], most[3]);
        const uint32_t mine = __float_as_uint(gt) & 0x7FFFFFFFu;
        const int eb = scale_exp(mz);
        eh = scale_exp(mh);
        ez = mine && mine < 0x7F800000u ? min(scale_exp(mine), eb + 100) : eb;
        own = ez - eb;
        if (threadIdx.x == 0) {
            a.zexp[n] = own;
            if (n == 0) {
                a.amax[0] = mh;
                a.amax[2] = mz;
            }
        }
    }
    const float rs = gt * exp2i(ez), rb = rs * exp2i(-own);
    if (threadIdx.x == 0) {
        a.nlse[n] = any ? -l * kLog2e : kNoLse;
        a.scale[n] = rs;
        a.scale_batch[n] = rb;
        a.to_own[n] = exp2i(own);
    }
    const auto put = [&](int k, int64_t id, float d, bool first) {
        a.ids[k * in.N + n] = (int)id;
        a.dzt[k * in.N + n] = d;
        if (a.blocks && id >= 0 && first)
            add_target(&a.blocks[(id >> 5) * a.nblocks + (n >> 5)], a.ents, (int)(n * t.K + k), (int)(n & 31) | (int)(id & 31) << 5, d);
    };
    if (DISTILL) {
        float* z = sm + t.K;
        entry_scores<RT, T>(in, n, t.K, q, ids, [&](int k, float x) { z[k] = x; });
        __syncthreads();
        for (int k = threadIdx.x; k < t.K; k += RT) {
            const int id = q[k] == 0.f ? -1 : ids[k];
            float qs = 0.f;
            bool first = true;
            if (id >= 0)
                for (int j = 0; j < t.K; ++j)
                    if (ids[j] == id && q[j] != 0.f) {
                        qs += q[j];
                        first &= j >= k;
                    }
            put(k, id, id >= 0 ? (expf(z[k] / t.T - l) - qs) * rb : 0.f, first);
        }
    } else if (warp == 0) {
        const float z = xid >= 0 ? warp_dot(h, w + xid * in.ldw, in.D, in.vec, lane) : 0.f;
        if (lane == 0) put(0, xid, xid >= 0 ? (expf(z - l) - 1.f) * rb : 0.f, true);
    }
    for (int i = threadIdx.x; i < in.Dp; i += RT) {  // columns past D are not read
        const int64_t at = n * in.Dp + i;
        const bool is = any && i < in.D;
        const float x = is && (sizeof(T) == 4 || a.hq) ? to_f32(h[i]) * exp2i(eh) : 0.f;
        const auto scaled = [&](uint16_t* to, int64_t rows, float y) {
            if (sizeof(T) == 4)
                split1(y, to[at], to[rows * in.Dp + at]);
            else
                to[at] = __half_as_ushort(__float2half_rn(y));
        };
        if (sizeof(T) == 4)
            scaled(a.hp, a.hrows, any ? x : 1.f);
        else
            a.hp[at] = is ? reinterpret_cast<const uint16_t*>(h)[i] : a.one;
        if (a.hq) scaled(a.hq, in.N, x * exp2i(-own));
    }
}

// Target entries of dz in columns [v0, v0 + P) of the current piece, a thread per entry (2 to
// 3 us a piece, launch included: nothing to gain).
__global__ void k_head_fix(const int* ids, const float* dzt, const float* to_own, int64_t total, int64_t rows, int v0, int P, uint16_t* dz,
                           int64_t pitch, int64_t piece, int fmt, int split) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= total) return;
    const int id = ids[i];
    if (id < v0 || id >= v0 + P) return;
    const int64_t n = i % rows, at = n * pitch + (id - v0);
    const float d = dzt[i] * to_own[n];
    const uint32_t w = pack16(d, 0.f, fmt);
    dz[at] = (uint16_t)w;
    if (split) dz[piece + at] = (uint16_t)pack16(d - unpack_f16(w).x, 0.f, 0);
}

// 8 elements of a row from column c on; columns past D are 0.
__device__ __forceinline__ void load8(const HeadIn& in, const float* src, int c, float (&x)[8]) {
    if (in.vec) {
        *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(src);
        *reinterpret_cast<float4*>(x + 4) = *(reinterpret_cast<const float4*>(src) + 1);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = c + j < in.D ? src[j] : 0.f;
    }
}
__device__ __forceinline__ uint32_t absmax8(const float (&x)[8], uint32_t m) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t b = __float_as_uint(x[j]) & 0x7FFFFFFFu;
        if (b < 0x7F800000u) m = max(m, b);
    }
    return m;
}
__device__ __forceinline__ void split8(const float (&x)[8], float sc, uint16_t* hi_at, uint16_t* lo_at) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float a = x[2 * j] * sc, b = x[2 * j + 1] * sc;
        hi[j] = pack_hi(a, b);
        const float2 h = unpack_f16(hi[j]);
        lo[j] = pack16(a - h.x, b - h.y, 0);
    }
    *reinterpret_cast<uint4*>(hi_at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(lo_at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}

// What a pass needs before its products, in one launch.
//   blockIdx.y = 0  the table packed in rows of Dp 16-bit elements (fp32: hi and lo
//                   pieces, a scale per block of 128 x 128 (k_head_fused to D = 64: 256 rows), its
//                   exponent in wexp: what the products take of the table between two
//                   read-outs, so that a scale is one factor there; a block is read once and
//                   kept in registers: 512 MB in and out for 10^6 x 64 in 89 us, 5.7 TB/s)
//   blockIdx.y = 1  forward: the hidden rows packed, a warp per row (fp32: a scale of each
//                   row's own, its exponent in row_exp); backward: the largest finite
//                   |grad| T and |hidden| over the rows that count, a share per block
//   blockIdx.y = 2  backward, k_head_fused: the blocks of targets cleared
struct PrepArgs {
    HeadIn in;
    uint16_t* wp;       // null: the table is read as it is
    int wrows;          // rows of a scale's block
    int* wexp;
    uint16_t* hp;       // null: not packed
    int* row_exp;
    Target t;
    int distill;
    const float* grad;
    uint32_t* shares;   // [2][kAmaxShares], |grad| T then |hidden|; null: no scales
    int hidden_max;     // |hidden|'s are wanted, else 0
    uint4* clear;
    int64_t nclear;
};

template <class T, int TH>  // TH threads; fp32: 4 groups of 8 elements a thread: 128 x 128, 256 x 64 (512 threads) or 128 x 64
__global__ void __launch_bounds__(TH, 1024 / TH) k_head_prep(const __grid_constant__ PrepArgs a) {
    const HeadIn& in = a.in;
    uint16_t* const wp = a.wp;
    uint16_t* const hp = a.hp;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __shared__ uint32_t red[2][TH / 32];
    if (blockIdx.y == 0) {
        if (!wp) return;
        const int g = in.Dp / 8;  // 8-element groups of a row
        const int64_t piece = in.V * in.Dp;
        if constexpr (sizeof(T) == 4) {
            const float* w = static_cast<const float*>(in.w);
            const int cb = (in.D + 127) / 128;  // blocks to a row of blocks
            const int rb = a.wrows;
            const int64_t all = (in.V + rb - 1) / rb * cb;
            for (int64_t blk = blockIdx.x; blk < all; blk += gridDim.x) {
                const int64_t v0 = blk / cb * rb;
                const int c0 = (int)(blk % cb) * 128;
                const int rows = (int)min((int64_t)rb, in.V - v0), bg = min(16, g - c0 / 8), total = rows * bg;
                const uint32_t inv = 65536u / bg + 1;  // i / bg for i < 2,048, bg <= 16
                float x[4][8];
                uint32_t m = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int i = threadIdx.x + q * TH, r = (int)(i * inv >> 16), c = c0 + (i - r * bg) * 8;
                    if (i < total) {
                        load8(in, w + (v0 + r) * in.ldw + c, c, x[q]);
                        m = absmax8(x[q], m);
                    }
                }
                m = __reduce_max_sync(0xffffffffu, m);
                if (lane == 0) red[0][warp] = m;
                __syncthreads();
#pragma unroll
                for (int q = 0; q < TH / 32; ++q) m = max(m, red[0][q]);
                __syncthreads();
                const int e = scale_exp(m);
                const float sc = exp2i(e);
                if (threadIdx.x == 0) a.wexp[blk] = e;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int i = threadIdx.x + q * TH, r = (int)(i * inv >> 16), c = c0 + (i - r * bg) * 8;
                    uint16_t* to = wp + (v0 + r) * in.Dp + c;
                    if (i < total) split8(x[q], sc, to, to + piece);
                }
            }
        } else {
            const uint16_t* w = static_cast<const uint16_t*>(in.w);
            const int64_t total = in.V * g;
            for (int64_t i = (int64_t)blockIdx.x * TH + threadIdx.x; i < total; i += (int64_t)gridDim.x * TH) {
                const int64_t r = i / g;
                const int c = (int)(i - r * g) * 8;
                const uint16_t* s = w + r * in.ldw + c;
                uint16_t x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = c + j < in.D ? s[j] : (uint16_t)0;
                *reinterpret_cast<uint4*>(wp + i * 8) = *reinterpret_cast<uint4*>(x);
            }
        }
    } else if (blockIdx.y == 1 && hp) {
        const int64_t piece = in.N * in.Dp;
        for (int64_t n = (int64_t)blockIdx.x * (TH / 32) + warp; n < in.N; n += (int64_t)gridDim.x * (TH / 32)) {
            const T* h = static_cast<const T*>(in.h) + n * in.ldh;
            if (sizeof(T) == 4) {
                uint32_t m = 0;
                for (int i = lane; i < in.D; i += 32) {
                    const uint32_t b = __float_as_uint(to_f32(h[i])) & 0x7FFFFFFFu;
                    if (b < 0x7F800000u) m = max(m, b);
                }
                const int e = scale_exp(__reduce_max_sync(0xffffffffu, m));
                if (lane == 0) a.row_exp[n] = e;
                for (int i = lane; i < in.Dp; i += 32) {
                    split1(i < in.D ? to_f32(h[i]) * exp2i(e) : 0.f, hp[n * in.Dp + i], hp[piece + n * in.Dp + i]);
                }
            } else {
                const uint16_t* s = reinterpret_cast<const uint16_t*>(h);
                for (int i = lane; i < in.Dp; i += 32) hp[n * in.Dp + i] = i < in.D ? s[i] : (uint16_t)0;
            }
        }
    } else if (blockIdx.y == 1) {
        if (!a.shares || blockIdx.x >= kAmaxShares) return;
        const int share = blockIdx.x, shares = min((int)gridDim.x, kAmaxShares);
        auto counts = [&](int64_t n) {
            if (!a.distill) return a.t.ids[n] != a.t.ignore && (uint64_t)a.t.ids[n] < (uint64_t)in.V;
            for (int64_t k = n * a.t.K; k < (n + 1) * a.t.K; ++k)
                if ((uint64_t)a.t.ids[k] < (uint64_t)in.V && a.t.logits[k] != -INFINITY) return true;
            return false;
        };
        uint32_t mz = 0, mh = 0;
        auto take = [](uint32_t& m, float x) {
            const uint32_t b = __float_as_uint(x) & 0x7FFFFFFFu;
            if (b < 0x7F800000u) m = max(m, b);
        };
        for (int64_t n = (int64_t)share * TH + threadIdx.x; n < in.N; n += (int64_t)shares * TH)
            if (counts(n)) take(mz, a.grad[n] * a.t.T);
        if (a.hidden_max)
            for (int64_t n = (int64_t)share * (TH / 32) + warp; n < in.N; n += (int64_t)shares * (TH / 32))
                if (counts(n)) {
                    const T* h = static_cast<const T*>(in.h) + n * in.ldh;
                    for (int i = lane; i < in.D; i += 32) take(mh, to_f32(h[i]));
                }
        mz = __reduce_max_sync(0xffffffffu, mz);
        mh = __reduce_max_sync(0xffffffffu, mh);
        if (lane == 0) {
            red[0][warp] = mz;
            red[1][warp] = mh;
        }
        __syncthreads();
        if (threadIdx.x < 2) {
            uint32_t m = 0;
            for (int q = 0; q < TH / 32; ++q) m = max(m, red[threadIdx.x][q]);
            a.shares[threadIdx.x * kAmaxShares + share] = m;
        }
        if (share == 0)  // shares that no block has
            for (int i = shares + threadIdx.x; i < kAmaxShares; i += TH) a.shares[i] = a.shares[kAmaxShares + i] = 0;
    } else {
        for (int64_t i = (int64_t)blockIdx.x * TH + threadIdx.x; i < a.nclear; i += (int64_t)gridDim.x * TH) a.clear[i] = make_uint4(0, 0, 0, 0);
    }
}

// Row id of dweight for every target id, from fp32 dz (Residue says why): a block per entry,
// the first one with its id.
template <class T>
__global__ void __launch_bounds__(256) k_head_target_rows(HeadIn in, const int* ids, const float* dzt, int K, const float* nlse, const float* scale, float c,
                                                          const uint32_t* amax_z, void* out, int type) {
    __shared__ float dz[kFewTargets];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, N = (int)in.N;
    const int id = ids[blockIdx.x];
    if (id < 0) return;
    static_assert(kFewTargets <= 256, "an entry per thread");
    if (__syncthreads_or(threadIdx.x < blockIdx.x && ids[threadIdx.x] == id)) return;
    const T* h = static_cast<const T*>(in.h);
    const T* w = static_cast<const T*>(in.w) + (int64_t)id * in.ldw;
    for (int n0 = warp * 4; n0 < N; n0 += 32) {
        const T* rows[4];
        float z[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) rows[u] = h + min(n0 + u, N - 1) * in.ldh;
        warp_dots<4>(w, rows, in.D, in.vec, lane, z);
        const float mine = lane & 2 ? (lane & 1 ? z[3] : z[2]) : (lane & 1 ? z[1] : z[0]);
        const int n = n0 + lane;
        if (lane < 4 && n < N) {
            float d = scale[n] != 0.f ? scale[n] * ex2(fmaf(mine, c, nlse[n])) : 0.f;
            for (int k = 0; k < K; ++k)
                if (ids[k * N + n] == id) d = dzt[k * N + n];
            dz[n] = d;
        }
    }
    __syncthreads();
    const Pow2 sc(-amax_exp(amax_z));
    for (int i = threadIdx.x; i < in.D; i += 256) {
        float s = 0.f;
#pragma unroll 8
        for (int n = 0; n < N; ++n) {
            const float x = to_f32(h[n * in.ldh + i]);
            s = dz[n] != 0.f ? fmaf(dz[n], x, s) : s;  // a row that does not count may hold anything
        }
        store_one(out, (int64_t)id * in.D + i, sc(s), type);
    }
}

// out[m, n] = the splits' partial sums, in split order, unscaled and rounded once.  A
// block takes 256 >> row_shift rows at a time, 1 << row_shift threads to a row, four
// columns a thread.  row_exp: exponents of the rows' scales, with those of amax_a and amax_b.
__global__ void __launch_bounds__(256) k_head_reduce(const float* partial, int splits, int64_t M, int64_t N, int64_t pp, OutArgs to, int row_shift,
                                                     const uint32_t* amax_a, const uint32_t* amax_b, const int* row_exp, Residue low) {
    const int e = amax_exp(amax_a) + amax_exp(amax_b);
    const int per = 1 << row_shift, c0 = ((int)threadIdx.x & (per - 1)) * 4;
    for (int64_t m = (int64_t)blockIdx.x * (256 >> row_shift) + (threadIdx.x >> row_shift); m < M; m += (int64_t)gridDim.x * (256 >> row_shift)) {
        const Pow2 sc(-e - (row_exp ? __ldg(&row_exp[m]) : 0));
        for (int64_t n = c0; n < N; n += per * 4) {
            const float* p = partial + m * pp + n;
            float4 s = *reinterpret_cast<const float4*>(p);
#pragma unroll 4
            for (int k = 1; k < splits; ++k) {
                const float4 y = *reinterpret_cast<const float4*>(p + (int64_t)k * M * pp);
                s = make_float4(s.x + y.x, s.y + y.y, s.z + y.z, s.w + y.w);
            }
            float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (low.K && n + j < N) v[j] += low(m, (int)n + j);
                v[j] = sc(v[j]);
            }
            const int64_t at = m * to.ldo + n;
            if (to.vec && n + 4 <= N) {
                if (to.type == TT_F32)
                    *reinterpret_cast<float4*>(static_cast<float*>(to.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
                else
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(to.out) + at) =
                        make_uint2(pack16(v[0], v[1], to.type == TT_BF16), pack16(v[2], v[3], to.type == TT_BF16));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n + j < N) store_one(to.out, at + j, v[j], to.type);
            }
        }
    }
}

// ---------------------------------------------------------------- host

namespace {

std::atomic<uint64_t> g_head_wait_ns{kHeadWaitNs};  // of the process: calls of other threads read it meanwhile

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
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

// A [pieces][rows][cols] array of 16-bit elements, rows `pitch` elements apart, read
// in boxes of 64 columns x box_rows rows; elements outside read as 0.
bool make_map(CUtensorMap* m, const void* p, int fmt, int64_t cols, int64_t rows, int pieces, int64_t pitch, int64_t piece, int box_rows) {
    EncodeTiled enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)pieces};
    const cuuint64_t strides[2] = {(cuuint64_t)pitch * 2, (cuuint64_t)(pieces > 1 ? piece : pitch * rows) * 2};
    const cuuint32_t box[3] = {kBK, (cuuint32_t)box_rows, 1}, one[3] = {1, 1, 1};
    return enc(m, fmt ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(p), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <int A, int B, int C, int D, int E>
struct KernelTag {};

// Workspace cut into 256-byte aligned blocks; with a null base only the size counts.
struct Arena {
    uint8_t* base;
    size_t used = 0;
    explicit Arena(void* p) : base(static_cast<uint8_t*>(p)) {}
    template <class T>
    T* get(int64_t n) {
        T* p = base ? reinterpret_cast<T*>(base + used) : nullptr;
        used += ((size_t)n * sizeof(T) + 255) / 256 * 256;
        return p;
    }
};

struct Operand {  // a 16-bit matrix the products read
    const uint16_t* p;
    int64_t rows, cols, pitch, piece;
};

template <int BN, bool AMN, bool BMN, int EPI, bool SPLIT>
bool run_gemm(const Operand& A, const Operand& B, GemmArgs a, int sms, int dev, cudaStream_t st) {
    CUtensorMap ma, mb;
    const int pieces = SPLIT ? 2 : 1;
    if (!make_map(&ma, A.p, a.fmt, A.cols, A.rows, pieces, A.pitch, A.piece, AMN ? 64 : 128)) return false;
    if (!make_map(&mb, B.p, a.fmt, B.cols, B.rows, pieces, B.pitch, B.piece, BMN ? 64 : BN)) return false;
    a.mtiles = (int)cdiv(a.M, 128);
    a.ntiles = (int)cdiv(a.N, BN);
    a.nstrips = (int)cdiv(a.ntiles, a.strip);
    a.units = EPI == kEpiOut ? (int64_t)a.mtiles * a.ntiles * a.splits : (int64_t)a.mtiles * a.nstrips;
    a.wait_ns = g_head_wait_ns.load(std::memory_order_relaxed);
    auto k = k_head_gemm<BN, AMN, BMN, EPI, SPLIT>;
    if (!allow_smem<KernelTag<BN, AMN, BMN, EPI, SPLIT>>(k, dev, GemmShape<BN, SPLIT>::kSmem)) return false;
    k<<<(unsigned)(a.units < sms ? a.units : sms), kGemmThreads, GemmShape<BN, SPLIT>::kSmem, st>>>(ma, mb, a);
    return cudaGetLastError() == cudaSuccess;
}

// Scores: 128-column tiles for fp32 (the ranges' sums stay in registers).
template <int EPI>
bool score_gemm(int bn, bool split, const Operand& A, const Operand& B, const GemmArgs& a, int sms, int dev, cudaStream_t st) {
    if constexpr (EPI != kEpiStatsLong)
        if (split) return run_gemm<128, false, false, EPI, true>(A, B, a, sms, dev, st);
    if (bn == 128) return run_gemm<128, false, false, EPI, false>(A, B, a, sms, dev, st);
    return run_gemm<256, false, false, EPI, false>(A, B, a, sms, dev, st);
}

// Gradient products.  AMN: dweight = dz^T hidden; else dhidden = dz weight.
template <bool AMN>
bool out_gemm(bool split, const Operand& A, const Operand& B, const GemmArgs& a, int sms, int dev, cudaStream_t st) {
    if (split) return run_gemm<128, AMN, true, kEpiOut, true>(A, B, a, sms, dev, st);
    return run_gemm<256, AMN, true, kEpiOut, false>(A, B, a, sms, dev, st);
}

template <int DT, bool SPLIT, int MODE>
bool run_fused(const Operand& X, const Operand& Y, FusedArgs a, int dev, cudaStream_t st) {
    using S = FusedShape<DT, SPLIT>;
    CUtensorMap mx, my;
    if (!make_map(&mx, X.p, a.fmt, X.cols, X.rows, S::PC, X.pitch, X.piece, 128)) return false;
    if (!make_map(&my, Y.p, a.fmt, Y.cols, Y.rows, S::PC, Y.pitch, Y.piece, S::BY)) return false;
    a.wait_ns = g_head_wait_ns.load(std::memory_order_relaxed);
    auto k = k_head_fused<DT, SPLIT, MODE>;
    if (!allow_smem<KernelTag<DT, SPLIT, MODE, 0, -1>>(k, dev, S::kSmem)) return false;
    k<<<(unsigned)a.runs.blocks, S::kThreads, S::kSmem, st>>>(mx, my, a);
    if (cudaGetLastError() != cudaSuccess) return false;
    const bool join_all = MODE == kDhidden && a.low.K;  // few rows: one x
    if (MODE == kLse || (a.runs.blocks == 1 && !join_all)) return true;
    const bool by_boundary = a.runs.xtiles >= a.runs.blocks && !join_all;
    const unsigned gx = (unsigned)(by_boundary ? a.runs.blocks - 1 : a.runs.xtiles);
    const unsigned gy = gx >= 256 ? 1 : (gx >= 64 ? 4 : (gx >= 16 ? 16 : 64));  // a block or more per SM
    constexpr bool dw = MODE == kDweight;  // fp32 dhidden is freed of its scales but the rows' already
    k_head_join<<<dim3(gx, gy), 128, 0, st>>>(a.runs, by_boundary, a.partial, a.to, a.X, a.D, SPLIT && !dw ? nullptr : a.amax_z,
                                              dw ? a.amax_h : nullptr, dw ? nullptr : a.zexp, a.low);
    return cudaGetLastError() == cudaSuccess;
}

template <int MODE>
bool fused(bool split, const Operand& X, const Operand& Y, const FusedArgs& a, int dev, cudaStream_t st) {
    if (a.D <= 64) return split ? run_fused<64, true, MODE>(X, Y, a, dev, st) : run_fused<64, false, MODE>(X, Y, a, dev, st);
    return split ? run_fused<128, true, MODE>(X, Y, a, dev, st) : run_fused<128, false, MODE>(X, Y, a, dev, st);
}

Runs make_runs(int64_t xrows, int64_t yrows, int by, int sms) {
    Runs r{(int)cdiv(xrows, 128), (int)cdiv(yrows, by), 0};
    r.blocks = (int)(r.total() < sms ? r.total() : sms);
    return r;
}

// Column tiles per strip: the fewest rounds of tiles over the blocks, and among the
// strips within 3% of that the longest (fewer pairs to join).
int choose_strip(int64_t mtiles, int64_t ntiles, int sms) {
    const int64_t g0 = cdiv(ntiles, 2048);
    auto rounds = [&](int64_t g) { return (double)cdiv(mtiles * cdiv(ntiles, g), sms) * g; };
    double least = 1e30;
    for (int64_t g = g0; g < g0 + 64 && g <= ntiles; ++g) least = fmin(least, rounds(g));
    int64_t best = g0;
    for (int64_t g = g0; g < g0 + 64 && g <= ntiles; ++g)
        if (rounds(g) <= 1.03 * least) best = g;
    return (int)best;
}

// K ranges of a product of `tiles` tiles and `chunks` K chunks: the shortest
// schedule, a unit counted as its chunks and 4 for its start and read-out, a split as what
// joining it costs: a load's share of its latency, or `elements` fp32 sums written and read.
// dhidden with its join, against a cost that knows no sizes: 3 x 32926 x 230 fp32 21 us
// (33), 305 x 46310 x 159 bf16 18 (23); from 100 x 100000 x 1024 on the same.
int choose_splits(int64_t tiles, int64_t chunks, int64_t elements, int sms) {
    const double join = 0.4 + 1.6 * fmin(1.0, (double)elements / (1 << 18));
    int best = 1;
    double bestc = 1e30;
    for (int s = 1; s <= sms && s <= chunks; ++s) {
        const double c = (double)cdiv(tiles * s, sms) * (cdiv(chunks, s) + 4) + (s > 1 ? join * s : 0.0);
        if (c < bestc) bestc = c, best = s;
    }
    return best;
}

struct Plan {
    HeadIn in;
    int type, fmt, split;    // split: fp32 operands in hi and lo pieces
    bool scaled;             // backward: dz is scaled (bf16 has fp32's range)
    int esize, sms, device;
    bool pack_h, pack_w;          // 16-bit copies of hidden and weight
    bool pack_h_fwd, pack_w_fwd;  // in the forward pass
    int bn_s;                // column tile of the score products
    int strip;
    int slots, per_slot;     // (maximum, sum) pairs per row: slots of per_slot
    bool few, few_wide;      // forward: scores by k_head_few, on few_blocks blocks
    int few_blocks, few_ksplit;
    size_t few_smem;
    bool fused_lse;          // scores by k_head_fused, its work shared as in
    Runs runs_lse, runs_dw, runs_dh;
    bool fused;              // backward: dz stays on the chip (k_head_fused)
    int64_t nblocks, vblocks;  // its 32 x 32 blocks
    int64_t hrows;             // rows of hidden's copy
    int64_t P;               // else: vocabulary piece
    int64_t pitch;           // its row pitch in dz
    int dh_splits, dw_splits;
    bool dh_direct;
    bool few_targets;        // their elements of dz are not left at 16 bits
    int64_t pp;              // row pitch of partial sums
};

bool aligned_rows(const void* p, int64_t ld, int esize) { return ((uintptr_t)p % 16 == 0) && (ld * esize % 16 == 0); }

// buffers: whether the call's buffers are all there; host checks come before any CUDA call
tt_status make_plan(const tt_head* hd, int K, bool buffers, Plan* p) {
    if (!hd) return TT_ERR_ARG;
    if (hd->dtype != TT_F32 && hd->dtype != TT_BF16 && hd->dtype != TT_F16) return TT_ERR_ARG;
    if (hd->rows < 0 || hd->dim < 1 || hd->vocab < 1 || K < 1 || K > kMaxTeacher) return TT_ERR_SHAPE;
    if (hd->rows > TT_HEAD_MAX_ROWS || hd->vocab > TT_HEAD_MAX_VOCAB || hd->dim > TT_HEAD_MAX_DIM) return TT_ERR_SHAPE;
    if (hd->rows * K > 2147483647ll) return TT_ERR_SHAPE;
    if (hd->hidden_stride < hd->dim || hd->weight_stride < hd->dim) return TT_ERR_SHAPE;
    p->type = hd->dtype;
    p->fmt = hd->dtype == TT_BF16;
    p->split = hd->dtype == TT_F32;
    p->scaled = hd->dtype != TT_BF16;
    p->esize = hd->dtype == TT_F32 ? 4 : 2;
    if (((uintptr_t)hd->hidden_dev | (uintptr_t)hd->weight_dev) % p->esize) return TT_ERR_ARG;
    if (!buffers) return TT_ERR_ARG;
    p->sms = head_sms(&p->device);
    if (p->sms <= 0) return TT_ERR_CUDA;
    HeadIn& in = p->in;
    in.h = hd->hidden_dev;
    in.w = hd->weight_dev;
    in.ldh = hd->hidden_stride;
    in.ldw = hd->weight_stride;
    in.N = hd->rows;
    in.V = hd->vocab;
    in.D = hd->dim;
    in.Dp = (in.D + 7) / 8 * 8;
    const bool ah = aligned_rows(in.h, in.ldh, p->esize), aw = aligned_rows(in.w, in.ldw, p->esize);
    in.vec = ah && aw && in.D % 8 == 0;
    p->pack_h = p->split || !ah;
    p->pack_w = p->split || !aw;
    p->pack_h_fwd = p->pack_h;
    p->pack_w_fwd = p->pack_w;
    const int64_t mt = cdiv(in.N, 128);
    // 256-column tiles read each operand row less often; 128-column tiles when the
    // wide ones would leave blocks without work
    p->bn_s = !p->split && mt * cdiv(in.V, 256) >= 2 * p->sms ? 256 : 128;
    p->strip = choose_strip(mt, cdiv(in.V, p->bn_s), p->sms);
    const int by = p->split && in.D > 64 ? 64 : 128;  // streamed rows per tile of k_head_fused
    p->runs_lse = Runs{};
    p->slots = (int)cdiv(cdiv(in.V, p->bn_s), p->strip);
    p->per_slot = kParts;
    // 16-bit types: with the hidden rows resident the scores are bound by the exponentials'
    // warps either way, and the 256-column tiles of k_head_gemm feed them faster (4096 x
    // 100003 x 64: 80 us, here 103); fp32 reads its two pieces of a tile once, not three
    // times (208 us there, 129 here)
    p->fused_lse = p->split && in.D <= 128 && mt * cdiv(in.V, by) < 1ll << 31;
    if (p->fused_lse && in.N > 0) {
        p->runs_lse = make_runs(in.N, in.V, by, p->sms);
        const int64_t shortest = p->runs_lse.total() / p->runs_lse.blocks;  // tiles of a run, rounded down
        p->slots = (int)(cdiv(p->runs_lse.ytiles, shortest) + 1);           // most runs that an x is in
        p->per_slot = 2 * (by / 64);
    }
    // few rows: a pass over the table as it is per eight of them, when its rows can be read
    // 4 bytes at a time.  Measured against the other kernels, rows x table: bf16 4 x 131072
    // x 4096 188 us (251), 8 x 131072 x 1024 61 (70), x 256 59 (59), but x 128 40 (34) and
    // 8 x 10^6 x 64 55 (38), where a tile's end outweighs its loads; fp32, which the others
    // copy in pieces first, 8 x 131072 x 1024 99 (432), 16 rows in two passes 192 (463),
    // 8 x 10^6 x 64 66 (144), 16 rows 125 (144).
    const int64_t chunks = cdiv((int64_t)in.D * p->esize, 64);
    p->few_smem = (size_t)(chunks * 512);
    p->few = in.N > 0 && in.N <= (p->split ? 16 : 8) && (p->split || in.D >= kFewMinDim) && (uintptr_t)in.w % 4 == 0 &&
             in.ldw * p->esize % 4 == 0 && (int64_t)in.D * p->esize % 4 == 0 && p->few_smem <= kFewSmem;
    p->few_wide = aw && (int64_t)in.D * p->esize % 16 == 0;
    if (p->few) {
        const int64_t tiles = cdiv(in.V, kFewRows), steps = cdiv(chunks, kFewStep);
        const int blocks = (p->few_smem <= 100 * 1024 ? 2 : 1) * p->sms;
        // warps share a tile's columns while the tiles alone would give a warp fewer than 4
        // of them, as long as each keeps two steps
        p->few_ksplit = 1;
        while (p->few_ksplit < kFewWarps && tiles * p->few_ksplit < 4ll * blocks * kFewWarps && steps >= 4 * p->few_ksplit) p->few_ksplit *= 2;
        const int64_t rounds = cdiv(tiles, kFewWarps / p->few_ksplit);
        p->few_blocks = (int)(rounds < blocks ? rounds : blocks);
        p->slots = p->few_blocks;
        p->per_slot = 1;
        p->fused_lse = false;
        p->runs_lse = Runs{};
        p->pack_h_fwd = p->pack_w_fwd = false;
    }
    // backward
    p->few_targets = !p->split && in.N * K <= kFewTargets;
    p->nblocks = cdiv(in.N, 32);
    p->vblocks = cdiv(in.V, 32);
    p->hrows = in.N;
    p->fused = in.D <= 128 && p->nblocks * p->vblocks <= kMaxBlocks;
    if (p->fused) {
        p->hrows = mt * 128;
        p->dh_splits = p->dw_splits = 1;
        p->dh_direct = true;
        if (in.N > 0) {
            p->runs_dh = make_runs(in.N, in.V, by, p->sms);
            p->runs_dw = make_runs(in.V, in.N, by, p->sms);
        }
        p->P = in.V;
        p->pitch = 0;
    } else {
        const int64_t vcap = cdiv(in.V, 64) * 64;
        int64_t P = in.N > 0 ? kDzBytes / (2 * (p->split ? 2 : 1) * in.N) : vcap;
        P = P / 1024 * 1024;
        if (P < 1024) P = 1024;
        if (P >= vcap) {
            P = vcap;
        } else {
            P = cdiv(cdiv(in.V, cdiv(in.V, P)), 256) * 256;  // pieces of near-equal size
        }
        p->P = P;
        p->pitch = P;
        const int bn = p->split ? 128 : 256;
        const int64_t nt = cdiv(in.D, bn), lastP = in.V - (cdiv(in.V, P) - 1) * P;
        p->dh_splits = choose_splits(mt * nt, cdiv(lastP, kBK), in.N * in.D, p->sms);
        p->dh_direct = p->dh_splits == 1 && in.V <= P && !p->few_targets;
        p->dw_splits = choose_splits(cdiv(P, 128) * nt, cdiv(in.N, kBK), P * in.D, p->sms);
    }
    p->pp = cdiv(in.D, 32) * 32;
    return TT_OK;
}

struct FwdWs {
    float2* part;
    uint16_t *hp, *wp;
    int *row_exp, *wexp;
};
size_t fwd_ws(const Plan& p, void* base, FwdWs* w) {
    Arena a(base);
    const int64_t pc = p.split ? 2 : 1;
    w->wexp = a.get<int>(p.split && p.pack_w_fwd ? cdiv(p.in.V, 128) * cdiv(p.in.D, 128) : 0);
    w->part = a.get<float2>(p.in.N * p.slots * p.per_slot);
    w->row_exp = a.get<int>(p.split && p.pack_h_fwd ? p.in.N : 0);
    w->hp = a.get<uint16_t>(p.pack_h_fwd ? pc * p.in.N * p.in.Dp : 0);
    w->wp = a.get<uint16_t>(p.pack_w_fwd ? pc * p.in.V * p.in.Dp : 0);
    return a.used;
}

struct BwdWs {
    uint32_t *amax, *shares;
    float *nlse, *scale, *scale_batch, *to_own, *joins, *dzt, *dh_part, *dw_part;
    int *zexp, *ids, *wexp;
    TargetBlock* blocks;
    TargetEntry* ents;
    uint16_t *hp, *hq, *wp, *dz;
};
size_t bwd_ws(const Plan& p, int K, void* base, BwdWs* w) {
    Arena a(base);
    const int64_t pc = p.split ? 2 : 1, nk = p.in.N * K;
    w->amax = a.get<uint32_t>(4);
    w->shares = a.get<uint32_t>(2 * kAmaxShares);
    w->wexp = a.get<int>(p.split ? cdiv(p.in.V, 128) * cdiv(p.in.D, 128) : 0);
    w->nlse = a.get<float>(cdiv(p.in.N, 128) * 128);
    w->scale = a.get<float>(cdiv(p.in.N, 128) * 128);
    w->scale_batch = p.scaled ? a.get<float>(cdiv(p.in.N, 128) * 128) : w->scale;
    w->to_own = a.get<float>(cdiv(p.in.N, 128) * 128);
    w->zexp = a.get<int>(p.scaled ? p.in.N : 0);
    w->ids = a.get<int>(nk);
    w->dzt = a.get<float>(nk);
    w->blocks = a.get<TargetBlock>(p.fused ? p.nblocks * p.vblocks : 0);
    w->ents = a.get<TargetEntry>(p.fused ? nk : 0);
    w->hp = a.get<uint16_t>(pc * p.hrows * p.in.Dp);
    w->hq = a.get<uint16_t>(p.scaled && !p.fused ? pc * p.in.N * p.in.Dp : 0);
    w->wp = a.get<uint16_t>(p.pack_w ? pc * p.in.V * p.in.Dp : 0);
    w->dz = a.get<uint16_t>(pc * p.in.N * p.pitch);
    w->joins = a.get<float>(p.fused ? (int64_t)p.sms * 2 * 128 * p.pp : 0);
    w->dh_part = a.get<float>(p.dh_direct ? 0 : (int64_t)p.dh_splits * p.in.N * p.pp);
    w->dw_part = a.get<float>(p.dw_splits > 1 ? (int64_t)p.dw_splits * p.P * p.pp : 0);
    return a.used;
}

unsigned grid_of(int64_t items, int per_block, int sms, int per_sm) {
    const int64_t b = cdiv(items, per_block);
    return (unsigned)(b < 1 ? 1 : (b > (int64_t)sms * per_sm ? (int64_t)sms * per_sm : b));
}

// 16 warps to a row instead of 4, an entry each: rows whose 4 warps would leave the SMs
// half empty, with entries enough for more.  bf16, 64 entries of width 1024: 200 rows 11 us
// a launch (4 warps: 14 to 20); fp32, 512 rows x 32 entries of width 128: 14 (4 warps: 9).
bool wide_rows(const Plan& p, int K) { return K >= 16 && p.in.N < 2ll * p.sms; }

bool launch_ok() { return cudaGetLastError() == cudaSuccess; }

template <class T>
bool launch_prep(const Plan& p, const PrepArgs& a, cudaStream_t st) {
    const int64_t w = !a.wp ? 0 : (p.split ? cdiv(p.in.V, a.wrows) * cdiv(p.in.D, 128) : cdiv(p.in.V * (p.in.Dp / 8), 256));
    const int64_t h = a.hp ? cdiv(p.in.N, 8) : (a.shares ? cdiv(p.in.N, 32) : 0), c = cdiv(a.nclear, 1024);
    const int64_t most = w > h ? (w > c ? w : c) : (h > c ? h : c);
    const dim3 grid(grid_of(most, 1, p.sms, 16), a.nclear ? 3 : (h ? 2 : 1));
    if (p.split && (p.in.Dp > 64 || a.wrows > 128))
        k_head_prep<T, 512><<<grid, 512, 0, st>>>(a);
    else
        k_head_prep<T, 256><<<grid, 256, 0, st>>>(a);
    return launch_ok();
}

GemmArgs gemm_args(const Plan& p, int* err) {
    GemmArgs a{};
    a.strip = 1;
    a.splits = 1;
    a.fmt = p.fmt;
    a.err = err;
    return a;
}

template <class T>
constexpr int type_of() { return sizeof(T) == 4 ? TT_F32 : (std::is_same<T, __half>::value ? TT_F16 : TT_BF16); }

template <class T>
bool run_few(const Plan& p, const FewArgs& a, cudaStream_t st) {
    auto k = p.few_wide ? k_head_few<T, type_of<T>(), true> : k_head_few<T, type_of<T>(), false>;
    if (!(p.few_wide ? allow_smem<KernelTag<type_of<T>(), 1, 0, 0, -2>>(k, p.device, kFewSmem)
                     : allow_smem<KernelTag<type_of<T>(), 0, 0, 0, -2>>(k, p.device, kFewSmem)))
        return false;
    k<<<(unsigned)p.few_blocks, kFewThreads, p.few_smem, st>>>(a);
    return cudaGetLastError() == cudaSuccess;
}

template <class T>
tt_status head_forward(const Plan& p, const Target& t, float* loss, float* lse, int* err, void* ws, size_t ws_bytes, cudaStream_t st) {
    const HeadIn& in = p.in;
    FwdWs w;
    if (fwd_ws(p, ws, &w) > ws_bytes) return TT_ERR_ARG;
    if (in.N == 0) return TT_OK;
    const bool distill = t.logits != nullptr;
    if (p.pack_h_fwd || p.pack_w_fwd) {
        PrepArgs a{};
        a.in = in;
        a.wp = p.pack_w_fwd ? w.wp : nullptr;
        a.wrows = p.fused_lse && in.D <= 64 ? 256 : 128;
        a.wexp = w.wexp;
        a.hp = p.pack_h_fwd ? w.hp : nullptr;
        a.row_exp = w.row_exp;
        if (!launch_prep<T>(p, a, st)) return TT_ERR_CUDA;
    }
    const Operand H{p.pack_h_fwd ? w.hp : static_cast<const uint16_t*>(in.h), in.N, in.D, p.pack_h_fwd ? in.Dp : in.ldh, in.N * in.Dp};
    const Operand W{p.pack_w_fwd ? w.wp : static_cast<const uint16_t*>(in.w), in.V, in.D, p.pack_w_fwd ? in.Dp : in.ldw, in.V * in.Dp};
    const int* row_exp = p.split ? w.row_exp : nullptr;
    bool ok;
    if (p.few) {
        FewArgs a{};
        a.w = in.w;
        a.ldh = in.ldh;
        a.ldw = in.ldw;
        a.V = in.V;
        a.D = in.D;
        a.chunks = (int)cdiv((int64_t)in.D * p.esize, 64);
        a.ksplit = p.few_ksplit;
        a.c = kLog2e / t.T;
        ok = true;
        for (int n0 = 0; ok && n0 < in.N; n0 += 8) {
            a.h = static_cast<const T*>(in.h) + n0 * in.ldh;
            a.N = (int)(in.N - n0 < 8 ? in.N - n0 : 8);
            a.part = w.part + (int64_t)n0 * p.slots;
            ok = run_few<T>(p, a, st);
        }
    } else if (p.fused_lse) {
        FusedArgs a{};
        a.X = in.N;
        a.Y = in.V;
        a.D = in.D;
        a.runs = p.runs_lse;
        a.slots = p.slots;
        a.fmt = p.fmt;
        a.err = err;
        a.wexp = w.wexp;
        a.row_exp = row_exp;
        a.ctemp = kLog2e / t.T;
        a.part = w.part;
        ok = fused<kLse>(p.split, H, W, a, p.device, st);
    } else {
        GemmArgs a = gemm_args(p, err);
        a.M = in.N;
        a.N = in.V;
        a.strip = p.strip;
        a.chunks = (int)cdiv(in.D, kBK);
        a.wexp = p.split ? w.wexp : nullptr;
        a.kb = (int)cdiv(in.D, 128);
        a.row_exp = row_exp;
        a.ctemp = kLog2e / t.T;
        a.part = w.part;
        ok = !p.split && a.chunks > kLongChunks ? score_gemm<kEpiStatsLong>(p.bn_s, false, H, W, a, p.sms, p.device, st)
                                                : score_gemm<kEpiStats>(p.bn_s, p.split, H, W, a, p.sms, p.device, st);
    }
    if (!ok) return TT_ERR_CUDA;
    if (distill && wide_rows(p, t.K))
        k_head_finish<T, true, kRowThreadsWide>
            <<<(unsigned)in.N, kRowThreadsWide, (size_t)t.K * 12, st>>>(in, t, w.part, p.slots, p.per_slot, p.runs_lse, loss, lse, err);
    else if (distill)
        k_head_finish<T, true, kRowThreads>
            <<<(unsigned)in.N, kRowThreads, (size_t)t.K * 12, st>>>(in, t, w.part, p.slots, p.per_slot, p.runs_lse, loss, lse, err);
    else
        k_head_finish<T, false, kRowThreads>
            <<<(unsigned)cdiv(in.N, kRowThreads / 32), kRowThreads, 0, st>>>(in, t, w.part, p.slots, p.per_slot, p.runs_lse, loss, lse, err);
    return launch_ok() ? TT_OK : TT_ERR_CUDA;
}

template <class T>
tt_status head_backward(const Plan& p, const Target& t, const float* lse, const float* grad, void* dh, void* dw, int* err, void* ws,
                        size_t ws_bytes, cudaStream_t st) {
    const HeadIn& in = p.in;
    BwdWs w;
    if (bwd_ws(p, t.K, ws, &w) > ws_bytes) return TT_ERR_ARG;
    if (in.N == 0) return cudaMemsetAsync(dw, 0, (size_t)in.V * in.D * p.esize, st) == cudaSuccess ? TT_OK : TT_ERR_CUDA;
    const bool distill = t.logits != nullptr;
    uint32_t* amax = p.scaled ? w.amax : nullptr;
    const int* zexp = p.scaled ? w.zexp : nullptr;
    const bool use_hq = p.scaled && !p.fused;
    TargetBlock* blocks = p.fused ? w.blocks : nullptr;
    if (amax || p.pack_w || blocks) {
        PrepArgs a{};
        a.in = in;
        a.wp = p.pack_w ? w.wp : nullptr;
        a.wrows = p.fused && in.D <= 64 ? 256 : 128;
        a.wexp = w.wexp;
        a.t = t;
        a.distill = distill;
        a.grad = grad;
        a.shares = amax ? w.shares : nullptr;
        a.hidden_max = p.split || use_hq;
        a.clear = reinterpret_cast<uint4*>(w.blocks);
        a.nclear = blocks ? p.nblocks * p.vblocks : 0;
        if (!launch_prep<T>(p, a, st)) return TT_ERR_CUDA;
    }
    const uint16_t one = p.type == TT_BF16 ? 0x3F80 : 0x3C00;
    const RowsArgs ra{lse,   grad,  w.shares, amax,           w.zexp, w.nlse, w.scale, w.scale_batch,             w.to_own,
                      w.ids, w.dzt, blocks,   (int)p.nblocks, w.ents, w.hp,   p.hrows, use_hq ? w.hq : nullptr, one,     err};
    const auto rows = [&](auto kernel, int threads) { kernel<<<(unsigned)p.hrows, threads, (size_t)t.K * 12, st>>>(in, t, ra); };
    if (distill && wide_rows(p, t.K))
        rows(k_head_rows<T, true, kRowThreadsWide>, kRowThreadsWide);
    else if (distill)
        rows(k_head_rows<T, true, kRowThreads>, kRowThreads);
    else
        rows(k_head_rows<T, false, kRowThreads>, kRowThreads);
    if (!launch_ok()) return TT_ERR_CUDA;
    const uint32_t *ah = amax, *az = amax ? amax + 2 : nullptr;
    const int64_t wpitch = p.pack_w ? in.Dp : in.ldw;
    const uint16_t* w0 = p.pack_w ? w.wp : static_cast<const uint16_t*>(in.w);
    const Operand H{w.hp, p.hrows, in.D, in.Dp, p.hrows * in.Dp};
    const auto dest = [&](void* out, float* partial) {
        OutArgs o{};
        o.out = out;
        o.ldo = in.D;
        o.type = p.type;
        o.vec = ((uintptr_t)out % 16 == 0) && ((int64_t)in.D * p.esize % 16 == 0);
        o.partial = partial;
        o.pp = p.pp;
        return o;
    };
    const Residue none{}, low = p.few_targets ? Residue{w.ids, w.dzt, w.to_own, in.w, in.ldw, in.N, t.K, p.fmt} : none;
    // the rows of dweight that the few targets name, again (k_head_target_rows)
    const auto target_rows = [&] {
        if constexpr (sizeof(T) == 2)
            if (p.few_targets)
                k_head_target_rows<T><<<(unsigned)(in.N * t.K), 256, 0, st>>>(in, w.ids, w.dzt, t.K, w.nlse, w.scale_batch, kLog2e / t.T, az, dw,
                                                                              p.type);
        return launch_ok();
    };
    const auto reduce = [&](const float* partial, int splits, int64_t rows, void* out, const uint32_t* ay, const int* row_exp,
                            const Residue& lw) {
        int shift = 3;
        while (shift < 8 && (4 << shift) < in.D) ++shift;
        // fp32's are in their own units already
        k_head_reduce<<<grid_of(rows, 256 >> shift, p.sms, 16), 256, 0, st>>>(partial, splits, rows, in.D, p.pp, dest(out, nullptr), shift,
                                                                            p.split ? nullptr : az, p.split ? nullptr : ay,
                                                                            p.split ? nullptr : row_exp, lw);
        return launch_ok();
    };
    if (p.fused) {
        const Operand W{w0, in.V, in.D, wpitch, in.V * in.Dp};
        FusedArgs a{};
        a.D = in.D;
        a.fmt = p.fmt;
        a.err = err;
        a.amax_h = p.split ? ah : nullptr;
        a.amax_z = az;
        a.zexp = zexp;
        a.to_own = w.to_own;
        a.wexp = w.wexp;
        a.ctemp = kLog2e / t.T;
        a.nlse = w.nlse;
        a.scale = w.scale_batch;
        a.blocks = w.blocks;
        a.ents = w.ents;
        a.ids = w.ids;
        a.dzt = w.dzt;
        a.K = t.K;
        a.rows = in.N;
        a.nblocks = (int)p.nblocks;
        a.vblocks = (int)p.vblocks;
        a.partial = w.joins;
        a.X = in.V;
        a.Y = in.N;
        a.runs = p.runs_dw;
        a.to = dest(dw, nullptr);
        if (!fused<kDweight>(p.split, W, H, a, p.device, st)) return TT_ERR_CUDA;
        a.X = in.N;
        a.Y = in.V;
        a.runs = p.runs_dh;
        a.scale = w.scale;
        a.to = dest(dh, nullptr);
        a.low = low;
        return fused<kDhidden>(p.split, H, W, a, p.device, st) && target_rows() ? TT_OK : TT_ERR_CUDA;
    }
    const Operand Hq{use_hq ? w.hq : w.hp, in.N, in.D, in.Dp, in.N * in.Dp};  // hrows is N here
    const int64_t npieces = cdiv(in.V, p.P), dz_piece = in.N * p.pitch;
    for (int64_t i = 0; i < npieces; ++i) {
        const int64_t v0 = i * p.P, P = in.V - v0 < p.P ? in.V - v0 : p.P;
        const Operand W{w0 + v0 * wpitch, P, in.D, wpitch, in.V * in.Dp};
        const Operand Z{w.dz, in.N, P, p.pitch, dz_piece};
        GemmArgs a = gemm_args(p, err);
        a.M = in.N;
        a.N = P;
        a.chunks = (int)cdiv(in.D, kBK);
        a.amax_a = p.split ? ah : nullptr;
        a.kb = (int)cdiv(in.D, 128);
        a.wexp = p.split ? w.wexp + v0 / 128 * a.kb : nullptr;  // a piece begins at a multiple of 256 rows
        a.ctemp = kLog2e / t.T;
        a.nlse = w.nlse;
        a.scale = w.scale;
        a.dz = w.dz;
        a.dz_pitch = p.pitch;
        a.dz_piece = dz_piece;
        if (!score_gemm<kEpiDz>(p.bn_s, p.split, H, W, a, p.sms, p.device, st)) return TT_ERR_CUDA;
        k_head_fix<<<(unsigned)cdiv(in.N * t.K, 256), 256, 0, st>>>(w.ids, w.dzt, w.to_own, in.N * t.K, in.N, (int)v0, (int)P, w.dz, p.pitch, dz_piece,
                                                                p.fmt, p.split);
        if (!launch_ok()) return TT_ERR_CUDA;

        GemmArgs b = gemm_args(p, err);  // dweight of the piece: [P][D] = dz^T H, the rows' scales evened out in H
        b.M = P;
        b.N = in.D;
        b.chunks = (int)cdiv(in.N, kBK);
        b.splits = p.dw_splits;
        b.amax_a = az;
        b.amax_b = ah;
        void* dwp = static_cast<uint8_t*>(dw) + (size_t)v0 * in.D * p.esize;
        b.to = dest(p.dw_splits > 1 ? nullptr : dwp, w.dw_part);
        if (!out_gemm<true>(p.split, Z, Hq, b, p.sms, p.device, st)) return TT_ERR_CUDA;
        if (p.dw_splits > 1 && !reduce(w.dw_part, p.dw_splits, P, dwp, ah, nullptr, none)) return TT_ERR_CUDA;

        GemmArgs c = gemm_args(p, err);  // the piece's share of dhidden: [N][D] += dz W
        c.M = in.N;
        c.N = in.D;
        c.chunks = (int)cdiv(P, kBK);
        c.splits = p.dh_splits;
        c.amax_a = az;
        c.row_exp = zexp;
        c.scale = w.scale;
        c.kb = (int)cdiv(in.D, 128);
        c.wexp = p.split ? w.wexp + v0 / 128 * c.kb : nullptr;
        c.to = dest(p.dh_direct ? dh : nullptr, w.dh_part);
        c.to.accumulate = i > 0;
        if (!out_gemm<false>(p.split, Z, W, c, p.sms, p.device, st)) return TT_ERR_CUDA;
    }
    if (!p.dh_direct && !reduce(w.dh_part, p.dh_splits, in.N, dh, nullptr, zexp, low)) return TT_ERR_CUDA;
    return target_rows() ? TT_OK : TT_ERR_CUDA;
}

tt_status forward_any(const tt_head* hd, const Target& t, float* loss, float* lse, int* err, void* ws, size_t n, tt_stream s) {
    Plan p;
    const bool buffers = hd && (hd->rows == 0 || (hd->hidden_dev && t.ids && loss && lse)) && hd->weight_dev &&
                         (ws || n == 0) && (uintptr_t)ws % 256 == 0;  // no rows may need no workspace
    const tt_status st = make_plan(hd, t.K, buffers, &p);
    if (st != TT_OK) return st;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(s);
    if (p.type == TT_F32) return head_forward<float>(p, t, loss, lse, err, ws, n, cs);
    if (p.type == TT_BF16) return head_forward<__nv_bfloat16>(p, t, loss, lse, err, ws, n, cs);
    return head_forward<__half>(p, t, loss, lse, err, ws, n, cs);
}

tt_status backward_any(const tt_head* hd, const Target& t, const float* lse, const float* grad, void* dh, void* dw, int* err, void* ws,
                       size_t n, tt_stream s) {
    Plan p;
    const bool buffers = hd && (hd->rows == 0 || (hd->hidden_dev && t.ids && lse && grad && dh)) && hd->weight_dev && dw && ws &&
                         (uintptr_t)ws % 256 == 0 && ((uintptr_t)dh | (uintptr_t)dw) % (hd->dtype == TT_F32 ? 4 : 2) == 0;
    const tt_status st = make_plan(hd, t.K, buffers, &p);
    if (st != TT_OK) return st;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(s);
    if (p.type == TT_F32) return head_backward<float>(p, t, lse, grad, dh, dw, err, ws, n, cs);
    if (p.type == TT_BF16) return head_backward<__nv_bfloat16>(p, t, lse, grad, dh, dw, err, ws, n, cs);
    return head_backward<__half>(p, t, lse, grad, dh, dw, err, ws, n, cs);
}

bool good_temp(float T) { return T > 0.f && T <= 1e4f && T >= 1e-4f; }

}  // namespace
}  // namespace ttemb

using namespace ttemb;

extern "C" {

int64_t tt_emb_head_workspace(const tt_head* head, int32_t teacher_k, int32_t backward) {
    Plan p;
    if (make_plan(head, teacher_k, true, &p) != TT_OK) return -1;
    if (backward) {
        BwdWs w;
        return (int64_t)bwd_ws(p, teacher_k, nullptr, &w);
    }
    FwdWs w;
    return (int64_t)fwd_ws(p, nullptr, &w);
}

tt_status tt_emb_xent_forward(const tt_head* head, const int64_t* targets_dev, int64_t ignore_index, float* loss_dev, float* lse_dev,
                              int32_t* err_dev, void* ws_dev, size_t ws_bytes, tt_stream stream) {
    const Target t{targets_dev, nullptr, ignore_index, 1, 1.f};
    return forward_any(head, t, loss_dev, lse_dev, err_dev, ws_dev, ws_bytes, stream);
}

tt_status tt_emb_xent_backward(const tt_head* head, const int64_t* targets_dev, int64_t ignore_index, const float* lse_dev,
                               const float* grad_loss_dev, void* grad_hidden_dev, void* grad_weight_dev, int32_t* err_dev, void* ws_dev,
                               size_t ws_bytes, tt_stream stream) {
    const Target t{targets_dev, nullptr, ignore_index, 1, 1.f};
    return backward_any(head, t, lse_dev, grad_loss_dev, grad_hidden_dev, grad_weight_dev, err_dev, ws_dev, ws_bytes, stream);
}

tt_status tt_emb_distill_forward(const tt_head* head, const int64_t* ids_dev, const float* logits_dev, int32_t teacher_k, float temperature,
                                 float* loss_dev, float* lse_dev, int32_t* err_dev, void* ws_dev, size_t ws_bytes, tt_stream stream) {
    if (!good_temp(temperature) || (head && head->rows > 0 && !logits_dev)) return TT_ERR_ARG;
    const Target t{ids_dev, logits_dev, -1, teacher_k, temperature};
    return forward_any(head, t, loss_dev, lse_dev, err_dev, ws_dev, ws_bytes, stream);
}

tt_status tt_emb_distill_backward(const tt_head* head, const int64_t* ids_dev, const float* logits_dev, int32_t teacher_k,
                                  float temperature, const float* lse_dev, const float* grad_loss_dev, void* grad_hidden_dev,
                                  void* grad_weight_dev, int32_t* err_dev, void* ws_dev, size_t ws_bytes, tt_stream stream) {
    if (!good_temp(temperature) || (head && head->rows > 0 && !logits_dev)) return TT_ERR_ARG;
    const Target t{ids_dev, logits_dev, -1, teacher_k, temperature};
    return backward_any(head, t, lse_dev, grad_loss_dev, grad_hidden_dev, grad_weight_dev, err_dev, ws_dev, ws_bytes, stream);
}

tt_status tt_emb_head_set_wait_limit(uint64_t ns) {
    g_head_wait_ns.store(ns, std::memory_order_relaxed);
    return TT_OK;
}

}  // extern "C"
