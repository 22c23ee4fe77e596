// tt_answers.cu -- losses of answers from the log probabilities of their tokens: the
// preference loss of pairs and the clipped policy loss, and their gradients.
//
// Both are sums over the tokens of a sequence, followed by a little arithmetic per sequence
// or pair; the gradient of a token is its own arithmetic times a number of its sequence.
// So they are streams: forward 9 (preference) or 13 to 17 bytes read a token (policy),
// backward the same (preference: the mask only) and 4 written.
//
// Tokens lie one behind the other and sequences are cut out of them by offsets that only
// the device knows.  Work is cut without looking at them: every sequence, and every multiple
// of K tokens, begins a piece, which ends where its sequence ends or at the next multiple of
// K.  So there are at most S + N / K pieces, each in one sequence and at most K tokens
// long, and piece u < S begins sequence u while piece S + c begins at token (c + 1) K (and is
// empty where a sequence begins there or none is).  A warp takes a piece, four tokens a
// lane and step; pieces of one sequence are joined in their order, so results repeat.
//
// Measured: 1,024 x 8,192 tokens, k3, an advantage each: 60 us both ways.  Under a profiler sums 30 us (143 MB; issue slots 65%
// and memory 62% busy, 90 instructions a token), numbers of the sequences 6, gradient 30 (55%, 66%, 77).  1,024 pairs, 4.2 M
// packed tokens: 25 us both ways where 55 MB take 8; which part of the way through a piece bounds it was not measured.
#include <cmath>

#include "tt_units.cuh"

namespace ttemb {

constexpr int kPieceMin = 8, kPieceMax = 11;  // log2 of K, tokens
constexpr int kAnswerWarps = 4;                   // pieces of a block
constexpr int kAnswerBlocks = 8;                  // of a multiprocessor
constexpr int kOneWarps = 32;                     // of the block that does a small call alone
constexpr int64_t kOneTokens = 8192, kOnePieces = 64;

// A sum in two floats, which keeps some 48 bits: every rounding of `hi` goes to `lo` (the exact
// error of an addition: D. E. Knuth, "The Art of Computer Programming", vol. 2, 4.2.2).  In doubles, and
// with 64-bit indexes, 8.4 M tokens of the policy loss took 201 us both ways, so and with 32-bit ones 107.
// What is added is a group of four tokens' terms, summed in fp32: at most 2 x 2^-24 of their magnitudes, where each
// term has an error of 2^-24 from its difference already; one addition to the two floats in place of four.
struct Long {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float x) {
        const float s = hi + x, b = s - hi;
        lo += (hi - (s - b)) + (x - b);
        hi = s;
    }
    __device__ __forceinline__ void add_lanes(int apart) {
        const float x = __shfl_xor_sync(0xffffffffu, hi, apart), y = __shfl_xor_sync(0xffffffffu, lo, apart);
        add(x);
        lo += y;
    }
    __device__ __forceinline__ void add(const Long& x) {
        add(x.hi);
        lo += x.lo;
    }
    __device__ __forceinline__ double value() const { return isfinite(hi) ? (double)hi + (double)lo : (double)hi; }
};

// Sums over a piece, and over a sequence.
struct __align__(16) Sums {
    Long a, b, c;  // preference: a = sum of log ratios; policy: L, k, d
    int count = 0, clipped = 0;
};
constexpr int64_t kSumsBytes = sizeof(Sums);
static_assert(sizeof(Sums) == 32, "layout of the workspace");

struct Two {  // a number in two pieces: hi + lo, lo at most half a unit of hi
    float hi, lo;
};

struct AnswerArgs {
    const float* logp;
    const float* ref;
    const uint8_t* mask;
    const int64_t* off;
    int64_t N, S, len;  // len: tokens of a sequence without offsets
    int shift;          // log2 of K
    int64_t chunks;     // pieces that begin at a multiple of K
    int average, vec;
    Sums* part;         // [S + chunks]
    int* err;
    float* grad;        // [N]
    const float* grad_loss;
    const int* counts;
    int* counts_out;
    float* loss;
    // preference
    int kind;
    int64_t pairs;
    Two beta, smoothing, rest;  // rest: 1 - smoothing
    double dbeta, dmargin, inverse_beta;
    float* margins;
    float* rewards;
    const float* margins_in;
    // policy
    const float* old;
    const float* adv;
    int per_token, sequence, kl;
    float low, high, dual;        // 1 - clip_low, 1 + clip_high, dual_clip
    Two tlow, thigh, tdual;  // their logarithms
    float kl_weight;
    float* kl_out;
    float* log_ratio;
    int* clipped;
    const float* log_ratio_in;
};

// The warp's number in its block, known to the compiler to be one value for the warp.
__device__ __forceinline__ int warp_id() { return __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0); }

struct Piece {
    int64_t s, b, e;  // sequence (S: behind the last one, -1: nothing), tokens [b, e)
};

__device__ __forceinline__ int64_t offset_at(const AnswerArgs& a, int64_t s) {
    if (!a.off) return s * a.len;
    const int64_t o = a.off[s];
    return o < 0 ? 0 : (o > a.N ? a.N : o);
}

// The sequence that holds token t, or S (behind the last one): the largest s with offset[s] <= t.
__device__ int64_t sequence_of(const AnswerArgs& a, int64_t t) {
    if (!a.off) {
        if (a.len == 0) return a.S;
        return a.N < 1ll << 31 ? (int64_t)((uint32_t)t / (uint32_t)a.len) : t / a.len;
    }
    const int lane = threadIdx.x & 31;
    int64_t lo = 0, hi = a.S;
    while (hi > lo) {  // 32 probes a step
        const int64_t step = (hi - lo + 32) / 32, at = lo + lane * step;
        const unsigned below = __ballot_sync(0xffffffffu, at <= hi && offset_at(a, at <= hi ? at : hi) <= t);
        const int n = __ffs(~below);  // 1 + how many of them in a row, from the first
        if (n <= 1 && below != 0xffffffffu) return lo;
        const int last = below == 0xffffffffu ? 31 : n - 2;
        lo += last * step;
        hi = min(hi, lo + step - 1);
    }
    return lo;
}

// Piece u; with_rest: the tokens behind the last sequence are sequence S.
__device__ __forceinline__ Piece piece_of(const AnswerArgs& a, int64_t u, bool with_rest) {
    const int64_t seqs = a.S + (with_rest ? 1 : 0);
    Piece p;
    if (u < seqs) {
        p.s = u;
        p.b = offset_at(a, u);
        p.e = u < a.S ? offset_at(a, u + 1) : a.N;
        p.e = min(p.e, ((p.b >> a.shift) + 1) << a.shift);
    } else {
        p.b = (u - seqs + 1) << a.shift;
        p.s = sequence_of(a, p.b);
        p.e = p.s < a.S ? offset_at(a, p.s + 1) : (with_rest ? a.N : p.b);
        p.e = min(p.e, p.b + ((int64_t)1 << a.shift));
        if (offset_at(a, p.s) >= p.b) p.e = p.b;  // begins there: has a piece of its own
    }
    return p;
}

// x against t for x = p - q without the rounding of the difference: -1, 0, 1.
__device__ __noinline__ int side_of(float p, float q, Two t) {
    const double x = (double)p - (double)q, y = (double)t.hi + (double)t.lo;
    return x > y ? 1 : (x < y ? -1 : 0);
}

// exp(y) - 1 - y = y^2 (1/2 + y/6 + ..) where the three nearly cancel, |y| <= 1: the first term left out is
// below 2^-27 of the sum.  From the highest power down.
constexpr int kTerms = 10;
__device__ constexpr float kSeries[kTerms] = {1.f / 39916800.f, 1.f / 3628800.f, 1.f / 362880.f, 1.f / 40320.f, 1.f / 5040.f,
                                              1.f / 720.f,      1.f / 120.f,     1.f / 24.f,     1.f / 6.f,     0.5f};
__device__ __forceinline__ float series(float y) {
    float s = kSeries[0];
#pragma unroll
    for (int i = 1; i < kTerms; ++i) s = fmaf(s, y, kSeries[i]);
    return s * y;
}
__device__ __noinline__ float exp_less_line(float y) {
    if (fabsf(y) <= 1.f) return series(y) * y;
    return y > 64.f ? expf(y) : expf(y) - 1.f - y;  // (infinite, not inf - inf)
}
__device__ __noinline__ float one_less_exp(float y) { return fabsf(y) <= 1.f ? fmaf(series(y), -y, -y) : 1.f - expf(y); }

// The clipped term of a token, x = p - q with d its rounded value: whether its ratio is beyond the bound, L, and dL/dx.
// The rounded d decides which side of a border x is on unless it is the rounded border itself: on_border.
struct Clipped {
    bool over;
    float term, slope;
};
// Bit 0: beyond the border on the side that A's sign names; bit 1: A < 0 and beyond dual_clip.
__device__ __noinline__ unsigned beyond_exactly(const AnswerArgs& a, bool up, float p, float q) {
    if (up) return side_of(p, q, a.thigh) > 0;
    return (side_of(p, q, a.tlow) < 0 ? 1u : 0u) | (side_of(p, q, a.tdual) > 0 ? 2u : 0u);
}
// A ratio: ex2.approx is good to 2 units, and rounding the product moves its exponent by 2^-24 |d|, as much
// as the rounding of d itself: what a more exact function would add to is lost in d before.
__device__ __forceinline__ float ratio_of(float d) { return ex2(d * kLog2e); }

// COUNT tokens at a time; one branch for the exact comparisons.
template <int COUNT>
__device__ __forceinline__ void clip_terms(const AnswerArgs& a, const float (&adv)[COUNT], const float (&d)[COUNT], const float (&p)[COUNT],
                                           const float (&q)[COUNT], Clipped (&c)[COUNT]) {
    bool border = false, dual[COUNT];
#pragma unroll
    for (int j = 0; j < COUNT; ++j) {
        const bool up = adv[j] > 0.f;
        const float past = up ? d[j] - a.thigh.hi : a.tlow.hi - d[j];
        c[j].over = past > 0.f;
        border = border || past == 0.f;
        dual[j] = false;
    }
    if (a.dual > 0.f) {
#pragma unroll
        for (int j = 0; j < COUNT; ++j) {
            dual[j] = !(adv[j] > 0.f) && d[j] > a.tdual.hi;
            border = border || d[j] == a.tdual.hi;
        }
    }
    if (border) {
#pragma unroll
        for (int j = 0; j < COUNT; ++j) {
            const unsigned b = beyond_exactly(a, adv[j] > 0.f, p[j], q[j]);
            c[j].over = b & 1;
            dual[j] = b & 2;
        }
    }
#pragma unroll
    for (int j = 0; j < COUNT; ++j) {
        const float r = ratio_of(d[j]), bound = adv[j] > 0.f ? a.high : (c[j].over ? a.low : a.dual);
        c[j].over = (c[j].over || dual[j]) && fabsf(adv[j]) > 0.f;  // no side without a sign: 0 (no bound), NaN (which stays in L and its slope)
        c[j].term = -adv[j] * (c[j].over ? bound : r);
        c[j].slope = c[j].over ? 0.f : c[j].term;
    }
}
__device__ __forceinline__ Clipped clip_term(const AnswerArgs& a, float adv, float d) {  // d as it is
    const float av[1] = {adv}, x[1] = {d}, zero[1] = {0.f};
    Clipped c[1];
    clip_terms<1>(a, av, x, x, zero, c);
    return c[0];
}

// k (slope: dk/dlogp) of two tokens' y = reference - logp.  The series of two at once.
__device__ __forceinline__ void kl_two(const AnswerArgs& a, float y0, float y1, bool slope, float& k0, float& k1) {
    if (a.kl != TT_KL_3) {
        const bool one = a.kl == TT_KL_1;
        k0 = one ? (slope ? 1.f : -y0) : (slope ? -y0 : 0.5f * y0 * y0);
        k1 = one ? (slope ? 1.f : -y1) : (slope ? -y1 : 0.5f * y1 * y1);
        return;
    }
    if (fmaxf(fabsf(y0), fabsf(y1)) <= 1.f) {
        k0 = k1 = kSeries[0];
#pragma unroll
        for (int i = 1; i < kTerms; ++i) fma2(k0, k1, y0, y1, kSeries[i], kSeries[i]);
        mul2(k0, k1, y0, y1);
        if (slope) {  // 1 - exp(y) = -y - y^2 (1/2 + ..)
            fma2(k0, k1, -y0, -y1, -y0, -y1);
        } else {
            mul2(k0, k1, y0, y1);
        }
    } else {
        k0 = slope ? one_less_exp(y0) : exp_less_line(y0);
        k1 = slope ? one_less_exp(y1) : exp_less_line(y1);
    }
}

// Four tokens of a piece, the first a multiple of 4 in the arrays.
struct Four {
    float lp[4], rf[4], od[4], ad[4];
    unsigned keep;  // bit 8 j + 7: token j is in the piece and counts
};
__device__ __forceinline__ bool kept(const Four& f, int j) { return f.keep & (0x80u << (8 * j)); }
__device__ __forceinline__ unsigned nonzero_bytes(unsigned m) { return (((m & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) | m) & 0x80808080u; }

// What of the arrays a pass reads.
struct Reads {
    bool lp, rf, od, ad;
};

// A group that is whole in the piece, at 16-byte boundaries.
__device__ __forceinline__ void load_whole(const AnswerArgs& a, int64_t i, Reads r, Four& f) {
    auto get = [&](const float* p, float (&v)[4]) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(p + i));
        v[0] = x.x;
        v[1] = x.y;
        v[2] = x.z;
        v[3] = x.w;
    };
    if (r.lp) get(a.logp, f.lp);
    if (r.rf) get(a.ref, f.rf);
    if (r.od) get(a.old, f.od);
    if (r.ad) get(a.adv, f.ad);
    f.keep = a.mask ? nonzero_bytes(__ldg(reinterpret_cast<const unsigned*>(a.mask + i))) : 0x80808080u;
}

// The same by way of shared memory: a lane's groups two steps ahead are on their way without a register for them.  Each
// lane copies and reads its own bytes, so nothing is waited for but its own copies.
struct __align__(16) Ahead {
    static constexpr int kStages = 3;
    float4 v[kStages][4][32];
    unsigned m[kStages][32];
    __device__ __forceinline__ void start(const AnswerArgs& a, int64_t i, Reads r, int stage, bool have) {
        const int lane = threadIdx.x & 31;
        if (have) {
            if (r.lp) cp16(&v[stage][0][lane], a.logp + i, true);
            if (r.rf) cp16(&v[stage][1][lane], a.ref + i, true);
            if (r.od) cp16(&v[stage][2][lane], a.old + i, true);
            if (r.ad) cp16(&v[stage][3][lane], a.adv + i, true);
            if (a.mask) cp4(&m[stage][lane], a.mask + i);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    __device__ __forceinline__ void take(const AnswerArgs& a, Reads r, int stage, Four& f) {
        const int lane = threadIdx.x & 31;
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        auto get = [&](int k, float (&x)[4]) {
            const float4 y = v[stage][k][lane];
            x[0] = y.x;
            x[1] = y.y;
            x[2] = y.z;
            x[3] = y.w;
        };
        if (r.lp) get(0, f.lp);
        if (r.rf) get(1, f.rf);
        if (r.od) get(2, f.od);
        if (r.ad) get(3, f.ad);
        f.keep = a.mask ? nonzero_bytes(m[stage][lane]) : 0x80808080u;
    }
};

// A piece's groups, a lane each at a time: those that are whole (`ahead`: the warp's own, or null), then the rest.
// take(f, first token of f)
template <class Take>
__device__ __forceinline__ void walk(const AnswerArgs& a, const Piece& p, Reads r, Ahead* ahead, Take take) {
    const int lane = threadIdx.x & 31;
    const int64_t from = a.vec ? (p.b + 3) & ~(int64_t)3 : p.e, to = a.vec ? p.e & ~(int64_t)3 : p.e;
    if (from < to) {
        const int n = (int)(to - from);
        int at = lane * 4;
        if (ahead) {
#pragma unroll
            for (int s = 0; s < Ahead::kStages - 1; ++s) ahead->start(a, from + at + s * 128, r, s, at + s * 128 < n);
            int stage = 0;
#pragma unroll 1
            for (; at < n; at += 128) {
                Four f;
                ahead->take(a, r, stage, f);
                // into the place that the step before has read
                ahead->start(a, from + at + (Ahead::kStages - 1) * 128, r, stage == 0 ? Ahead::kStages - 1 : stage - 1, at + (Ahead::kStages - 1) * 128 < n);
                stage = stage + 1 == Ahead::kStages ? 0 : stage + 1;
                take(f, from + at);
            }
        } else {
#pragma unroll 1
            for (; at < n; at += 128) {
                Four f;
                load_whole(a, from + at, r, f);
                take(f, from + at);
            }
        }
    }
    // groups that are not whole: all where the arrays are not aligned, else the first and the last
    const int64_t first = p.b & ~(int64_t)3, last = (p.e - 1) & ~(int64_t)3;
    for (int64_t i = a.vec ? (lane == 0 ? first : last) : first + lane * 4; i <= last; i += a.vec ? p.e : 128) {
        if (i >= from && i + 4 <= to) break;
        if (a.vec && (lane > 1 || (lane == 1 && first == last))) break;
        Four f;
        f.keep = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t k = i + j;
            if (k < p.b || k >= p.e) continue;
            if (r.lp) f.lp[j] = __ldg(a.logp + k);
            if (r.rf) f.rf[j] = __ldg(a.ref + k);
            if (r.od) f.od[j] = __ldg(a.old + k);
            if (r.ad) f.ad[j] = __ldg(a.adv + k);
            if (!a.mask || __ldg(a.mask + k)) f.keep |= 0x80u << (8 * j);
        }
        take(f, i);
    }
}

template <bool POLICY>
__device__ __forceinline__ Sums sum_piece(const AnswerArgs& a, const Piece& p, Ahead* ahead) {
    Sums s;
    if (p.b < p.e) {
        const bool ref = a.ref != nullptr, per_token = POLICY && a.per_token, clip = POLICY && !a.sequence;
        const float seq_adv = POLICY && !a.per_token ? __ldg(a.adv + p.s) : 0.f;
        walk(a, p, Reads{true, ref, POLICY, per_token}, ahead, [&](const Four& f, int64_t) {
            s.count += __popc(f.keep);
            float x[4];
            if constexpr (!POLICY) {
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = kept(f, j) ? (ref ? f.lp[j] - f.rf[j] : f.lp[j]) : 0.f;
                s.a.add((x[0] + x[1]) + (x[2] + x[3]));
            } else {
                float d[4], adv[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) d[j] = f.lp[j] - f.od[j];
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = kept(f, j) ? d[j] : 0.f;
                s.c.add((x[0] + x[1]) + (x[2] + x[3]));
                if (clip) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) adv[j] = per_token ? f.ad[j] : seq_adv;
                    Clipped c[4];
                    clip_terms<4>(a, adv, d, f.lp, f.od, c);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[j] = kept(f, j) ? c[j].term : 0.f;
                        s.clipped += kept(f, j) && c[j].over;
                    }
                    s.a.add((x[0] + x[1]) + (x[2] + x[3]));
                }
                if (ref) {
                    kl_two(a, f.rf[0] - f.lp[0], f.rf[1] - f.lp[1], false, x[0], x[1]);
                    kl_two(a, f.rf[2] - f.lp[2], f.rf[3] - f.lp[3], false, x[2], x[3]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] = kept(f, j) ? x[j] : 0.f;
                    s.b.add((x[0] + x[1]) + (x[2] + x[3]));
                }
            }
        });
    }
    __syncwarp();
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        s.a.add_lanes(o);
        if (POLICY) {
            s.b.add_lanes(o);
            s.c.add_lanes(o);
        }
    }
    s.count = __reduce_add_sync(0xffffffffu, s.count);
    if (POLICY) s.clipped = __reduce_add_sync(0xffffffffu, s.clipped);
    return s;
}

// All pieces of sequence s, by half a warp; each of its lanes has the result.  (Both halves call it.)
__device__ __forceinline__ Sums sum_sequence(const AnswerArgs& a, const Sums* part, int64_t s) {
    const int64_t b = offset_at(a, s), e = offset_at(a, s + 1), c0 = b >> a.shift, c1 = e > b ? (e - 1) >> a.shift : c0;
    Sums t;
    for (int64_t c = c0 + (threadIdx.x & 15); c <= c1; c += 16) {  // the piece of the sequence in [c K, (c + 1) K)
        const Sums x = part[c == c0 ? s : a.S + c - 1];
        t.a.add(x.a);
        t.b.add(x.b);
        t.c.add(x.c);
        t.count += x.count;
        t.clipped += x.clipped;
    }
#pragma unroll
    for (int o = 8; o; o >>= 1) {
        t.a.add_lanes(o);
        t.b.add_lanes(o);
        t.c.add_lanes(o);
        t.count += __shfl_xor_sync(0xffffffffu, t.count, o);
        t.clipped += __shfl_xor_sync(0xffffffffu, t.clipped, o);
    }
    return t;
}

// 1 / n (1 for none) to some 2^-48: a step of Newton's from the fp32 quotient costs two double operations, a division dozens.
__device__ __forceinline__ double inverse_of(int n) {
    const double d = n > 0 ? (double)n : 1.0, r = (double)(1.f / (float)(n > 0 ? n : 1));
    return fma(r, fma(-d, r, 1.0), r);
}

// Arithmetic of a pair's few numbers in two floats, so that its loss and its tokens' gradient are rounded once (sums and products with
// their exact errors: T. J. Dekker, "A floating-point technique for extending the available precision", 1971).  Written so that no
// product is fused with what is added to it, where the sum's own rounding is asked for.
__device__ __forceinline__ Two two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), c = __fadd_rn(s, -a);
    return {s, __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -c)), __fadd_rn(b, -c))};
}
__device__ __forceinline__ Two two_norm(float hi, float lo) {  // |lo| is far below |hi|
    const float s = __fadd_rn(hi, lo);
    return {s, __fadd_rn(lo, -__fadd_rn(s, -hi))};
}
__device__ __forceinline__ Two two_add(Two a, Two b) {
    const Two s = two_sum(a.hi, b.hi);
    return two_norm(s.hi, s.lo + (a.lo + b.lo));
}
__device__ __forceinline__ Two two_mul(Two a, Two b) {
    const float p = __fmul_rn(a.hi, b.hi);
    return two_norm(p, fmaf(a.hi, b.lo, fmaf(a.lo, b.hi, fmaf(a.hi, b.hi, -p))));
}
__device__ __forceinline__ Two two_div(Two a, Two b) {
    const float q = a.hi / b.hi, r = fmaf(-q, b.lo, fmaf(-q, b.hi, a.hi) + a.lo);
    return two_norm(q, r / b.hi);
}

// exp(x), x <= 0, to some 2^-26: with x = n log 2 + r it is 2^n (1 + r + r^2 (1/2 + ..)), of which only the last term is a plain fp32 number.
__device__ Two two_exp(float x) {
    if (!(x > -80.f)) return {expf(x), 0.f};
    constexpr double kLn2 = 0.69314718055994531;
    constexpr float kHi = (float)kLn2, kLo = (float)(kLn2 - (double)kHi);
    const float n = rintf(x * kLog2e), p = __fmul_rn(n, kHi);
    const Two d = two_sum(x, -p), r = two_norm(d.hi, d.lo - fmaf(n, kLo, fmaf(n, kHi, -p)));
    const Two s = two_sum(1.f, r.hi), e = two_norm(s.hi, s.lo + (r.lo + series(r.hi) * r.hi));
    const float scale = __int_as_float((127 + (int)n) << 23);
    return {e.hi * scale, e.lo * scale};
}
// log(1 + e), 0 <= e <= 1, as good: its series, or a step of Newton's from the fp32 function.
__device__ Two two_log1p(Two e) {
    if (!(e.hi > 0.0625f)) {
        float q = 1.f / 9.f;
#pragma unroll
        for (int k = 8; k >= 2; --k) q = fmaf(-q, e.hi, 1.f / (float)k);
        const Two s = two_sum(e.hi, __fmul_rn(__fmul_rn(-q, e.hi), e.hi));
        return two_norm(s.hi, s.lo + e.lo);
    }
    const float y = log1pf(e.hi);
    const Two d = two_sum(1.f, e.hi), p = two_mul({d.hi, d.lo + e.lo}, two_exp(-y));
    return two_norm(y, (p.hi - 1.f) + p.lo);
}

// sigma(h) and sigma(-h).
__device__ void sigmoids(float h, Two& up, Two& down) {
    const Two e = two_exp(-fabsf(h)), s = two_sum(1.f, e.hi), d = {s.hi, s.lo + e.lo};
    const Two large = two_div({1.f, 0.f}, d), small = two_div(e, d);
    up = h < 0.f ? small : large;
    down = h < 0.f ? large : small;
}
__device__ __forceinline__ Two sigmoid_slope(const AnswerArgs& a, Two up, Two down) {
    const Two d = two_mul(a.rest, down);
    return two_add(two_mul(a.smoothing, up), {-d.hi, -d.lo});
}

// g beta dloss/dh / n of a pair, of the margin that the forward call wrote.
__device__ float pref_weight(const AnswerArgs& a, float g, float h, int n) {
    const Two count = two_sum((float)(n & ~4095), (float)(n & 4095));
    Two v;
    float plain;  // where a number is not finite, two pieces of it are not
    if (a.kind == TT_PREF_HINGE) {
        const float slope = isnan(h) ? h : (h < 1.f ? -1.f : 0.f);  // a NaN stays in the gradient too
        v = two_mul(a.beta, {slope, 0.f});
        plain = slope * a.beta.hi;
    } else if (a.kind == TT_PREF_SQUARED) {
        const Two s = two_sum(h, -0.5f);
        v = two_div({2.f * s.hi, 2.f * s.lo}, a.beta);
        plain = 2.f * (h - 0.5f) / a.beta.hi;
    } else {
        Two up, down;
        sigmoids(h, up, down);
        const Two slope = sigmoid_slope(a, up, down);
        v = two_mul(slope, a.beta);
        plain = slope.hi * a.beta.hi;
    }
    v = two_div(two_mul(v, {g, 0.f}), count);
    return isfinite(v.hi) ? v.hi : g * plain / (float)n;
}

// The numbers of pair u (preference: a half of the warp for each answer) or of sequences 2 u and 2 u + 1 (policy), by a warp.
template <bool POLICY>
__device__ void finish_two(const AnswerArgs& a, const Sums* part, int64_t u) {
    const int half = (threadIdx.x >> 4) & 1;
    const int64_t s = POLICY ? 2 * u + half : u + half * a.pairs;
    const Sums t = sum_sequence(a, part, s < a.S ? s : a.S - 1);
    const bool lead = (threadIdx.x & 15) == 0 && s < a.S;
    if (POLICY) {
        if (!lead) return;
        const double inverse = inverse_of(t.count), share = a.average ? inverse : 1.0;
        const float x = (float)(t.c.value() * inverse);
        double term = t.a.value();
        int over = t.clipped;
        if (a.sequence) {
            const Clipped c = clip_term(a, a.adv[s], x);
            term = t.count > 0 ? (double)c.term * t.count : 0.0;
            over = c.over ? t.count : 0;
        }
        const double k = share * t.b.value();
        a.log_ratio[s] = x;
        a.kl_out[s] = (float)k;
        a.loss[s] = (float)(share * term + (a.kl_weight != 0.f ? a.kl_weight * k : 0.0));
        a.counts_out[s] = t.count;
        a.clipped[s] = over;
    } else {
        const double mine = a.dbeta * t.a.value() * (a.average ? inverse_of(t.count) : 1.0), other = __shfl_xor_sync(0xffffffffu, mine, 16);
        if (!lead) return;
        a.rewards[s] = (float)mine;
        a.counts_out[s] = t.count;
        if (half) return;
        const double margin = mine - other - a.dmargin;
        const float h = (float)margin;
        float loss;
        if (a.kind == TT_PREF_SIGMOID) {
            // -log sigma(h) = log(1 + exp(-|h|)) + max(-h, 0); of h's first piece, and the slope times the second
            if (isfinite(h)) {
                Two up, down, s = two_log1p(two_exp(-fabsf(h)));
                s = two_add(s, two_mul(h < 0.f ? a.rest : a.smoothing, {fabsf(h), 0.f}));
                sigmoids(h, up, down);
                loss = s.hi + fmaf(sigmoid_slope(a, up, down).hi, (float)(margin - (double)h), s.lo);
            } else {
                loss = isnan(h) ? h : (h < 0.f || a.smoothing.hi > 0.f ? INFINITY : 0.f);
            }
        } else if (a.kind == TT_PREF_HINGE) {
            loss = isnan(h) ? h : (float)fmax(1.0 - margin, 0.0);
        } else {
            const double v = margin - 0.5;
            loss = (float)(v * a.inverse_beta * (v * a.inverse_beta));
        }
        a.loss[u] = loss;
        a.margins[u] = h;
    }
}

__device__ __forceinline__ void check_offsets(const AnswerArgs& a, int64_t u) {  // by one lane, u < S
    if (!a.off || !a.err) return;
    const int64_t b = a.off[u], e = a.off[u + 1];
    if (b < 0 || e < b || e > a.N || e - b > 0x7FFFFFFF || (u == 0 && b != 0)) atomicOr(a.err, kErrOffsets);
}

template <bool POLICY>
__global__ void __launch_bounds__(kAnswerWarps * 32, kAnswerBlocks) k_answer_sums(const __grid_constant__ AnswerArgs a) {
    const int64_t u = (int64_t)blockIdx.x * kAnswerWarps + warp_id();
    __shared__ Ahead ahead[kAnswerWarps];
    pdl_launch_dependents();
    if (u >= a.S + a.chunks) return;
    const Sums s = sum_piece<POLICY>(a, piece_of(a, u, false), &ahead[warp_id()]);
    if ((threadIdx.x & 31) == 0) {
        a.part[u] = s;
        if (u < a.S) check_offsets(a, u);
    }
}

template <bool POLICY>
__global__ void __launch_bounds__(kAnswerWarps * 32) k_answer_finish(const __grid_constant__ AnswerArgs a) {
    const int64_t u = (int64_t)blockIdx.x * kAnswerWarps + warp_id();
    pdl_wait();
    if (u < (POLICY ? (a.S + 1) / 2 : a.pairs)) finish_two<POLICY>(a, a.part, u);
}

// A small call: both steps in one block.
template <bool POLICY>
__global__ void __launch_bounds__(kOneWarps * 32) k_answer_one(const __grid_constant__ AnswerArgs a) {
    __shared__ __align__(16) uint8_t space[kOnePieces * sizeof(Sums)];
    Sums* part = reinterpret_cast<Sums*>(space);
    const int warp = warp_id();
    for (int64_t u = warp; u < a.S + a.chunks; u += kOneWarps) {
        const Sums s = sum_piece<POLICY>(a, piece_of(a, u, false), nullptr);
        if ((threadIdx.x & 31) == 0) {
            part[u] = s;
            if (u < a.S) check_offsets(a, u);
        }
    }
    __syncthreads();
    for (int64_t u = warp; u < (POLICY ? (a.S + 1) / 2 : a.pairs); u += kOneWarps) finish_two<POLICY>(a, part, u);
}

template <bool POLICY>
__global__ void __launch_bounds__(kAnswerWarps * 32, kAnswerBlocks) k_answer_grad(const __grid_constant__ AnswerArgs a) {
    const int64_t u = (int64_t)blockIdx.x * kAnswerWarps + warp_id();
    __shared__ Ahead ahead[kAnswerWarps];
    if (u >= a.S + 1 + a.chunks) return;
    const Piece p = piece_of(a, u, true);
    if (p.b >= p.e) return;
    const bool in = p.s < a.S;
    float g = 0.f, adv = 0.f, seq_slope = 0.f;
    if (in) {
        const int n = a.average ? max(a.counts[p.s], 1) : 1;
        if (POLICY) {
            g = a.grad_loss[p.s] / (float)n;
            if (!a.per_token) adv = a.adv[p.s];
            if (a.sequence) {
                const float x = a.log_ratio_in[p.s];
                seq_slope = clip_term(a, adv, x).slope;
            }
        } else {
            const bool chosen = p.s < a.pairs;
            const int64_t pair = chosen ? p.s : p.s - a.pairs;
            g = pref_weight(a, a.grad_loss[pair], a.margins_in[pair], n);
            if (!chosen) g = -g;
        }
    }
    const bool kl = POLICY && in && a.ref && a.kl_weight != 0.f, ratio = POLICY && in && !a.sequence;
    const bool per_token = ratio && a.per_token;
    walk(a, p, Reads{kl || ratio, kl, ratio, per_token}, &ahead[warp_id()], [&](const Four& f, int64_t at) {
        float v[4];
        if (POLICY) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = seq_slope;
            if (ratio) {
                float adv4[4], d[4];
                Clipped c[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    adv4[j] = per_token ? f.ad[j] : adv;
                    d[j] = f.lp[j] - f.od[j];
                }
                clip_terms<4>(a, adv4, d, f.lp, f.od, c);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = c[j].slope;
            }
            if (kl) {
                float k[4];
                kl_two(a, f.rf[0] - f.lp[0], f.rf[1] - f.lp[1], true, k[0], k[1]);
                kl_two(a, f.rf[2] - f.lp[2], f.rf[3] - f.lp[3], true, k[2], k[3]);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = fmaf(a.kl_weight, k[j], v[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = in && kept(f, j) ? (POLICY ? g * v[j] : g) : 0.f;
        if (a.vec && at >= p.b && at + 4 <= p.e) {
            *reinterpret_cast<float4*>(a.grad + at) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
            for (int j = 0; j < 4; ++j)
                if (at + j >= p.b && at + j < p.e) a.grad[at + j] = v[j];
        }
    });
}

namespace {

tt_status answer_sizes(int64_t tokens, int64_t sequences) {
    return tokens < 0 || sequences < 0 || tokens > TT_ANSWERS_MAX_TOKENS || sequences > TT_ANSWERS_MAX_SEQUENCES ? TT_ERR_SHAPE : TT_OK;
}

// log2 of the tokens of a piece.  Short ones spread over the device, and even out what its last blocks have to do; long
// ones cost fewer sums to write and join.  The policy loss has more to do per token.  Both ways, us, in pieces of 256 / 512 / 1,024 / 2,048 tokens:
//   policy       2^20 tokens 14 / 14 / 16 / 14, 2^21 22 / 21 / 21 / 25, 2^22 37 / 34 / 35 / 35, 2^23 63 / 60 / 62 / 69, 2^25 226 / 197 / 197 / 202
//   preference   2^20 9.7 / 8.3 / 8.5 / 8.2, 2^21 13 / 11 / 10 / 11, 2^22 23 / 20 / 20 / 17, 2^23 38 / 32 / 29 / 32, 2^25 134 / 109 / 101 / 103
// The limits keep within a tenth of the best of these, the preference loss's within a fifth (2^20, 2^22).
int piece_shift(int64_t tokens, bool policy) {
    int k = kPieceMin;
    while (k < kPieceMax && tokens >> k > (policy ? 16384 : 4096)) ++k;
    return k;
}

// One launch, and no workspace: a forward call of 8,192 tokens takes 25 us of host time (policy; preference 21), in two launches 30 (26).
// The device's time is below that: both ways, policy, 512 tokens 6.2 us (6.3 in two launches), 2,048 7.9 (7.2), 8,192 11.8 (7.2); preference 4.8 (5.5),
// 5.2 (5.5), 7.2 (5.8).
bool in_one_block(int64_t tokens, int64_t pieces) { return tokens <= kOneTokens && pieces <= kOnePieces; }

tt_status fill_answers(const tt_answers* in, bool policy, AnswerArgs* a) {
    if (!in) return TT_ERR_ARG;
    const tt_status st = answer_sizes(in->tokens, in->sequences);
    if (st != TT_OK) return st;
    if (!in->offsets_dev && (in->sequences ? in->tokens % in->sequences : in->tokens)) return TT_ERR_SHAPE;
    if ((uintptr_t)in->offsets_dev % 8 || (uintptr_t)in->logp_dev % 4 || (uintptr_t)in->reference_dev % 4) return TT_ERR_ARG;
    a->logp = in->logp_dev;
    a->ref = in->reference_dev;
    a->mask = in->mask_dev;
    a->off = in->offsets_dev;
    a->N = in->tokens;
    a->S = in->sequences;
    a->len = in->sequences ? in->tokens / in->sequences : 0;
    a->shift = piece_shift(in->tokens, policy);
    a->chunks = in->tokens > 0 ? (in->tokens - 1) >> a->shift : 0;
    a->average = in->average != 0;
    if (!a->off && a->len > 0x7FFFFFFF) return TT_ERR_SHAPE;  // counts are int32
    return TT_OK;
}

Two split(double x) {
    const float hi = (float)x;
    return {hi, (float)(x - hi)};
}

tt_status fill_preference(const tt_preference* how, AnswerArgs* a) {
    if (!how || how->kind < TT_PREF_SIGMOID || how->kind > TT_PREF_SQUARED) return TT_ERR_ARG;
    if (!(how->beta > 0.0 && how->beta <= 1e6) || !(how->label_smoothing >= 0.0 && how->label_smoothing < 1.0) || !std::isfinite(how->margin))
        return TT_ERR_ARG;
    if (how->kind != TT_PREF_SIGMOID && how->label_smoothing != 0.0) return TT_ERR_ARG;
    if (a->S % 2) return TT_ERR_SHAPE;
    a->kind = how->kind;
    a->pairs = a->S / 2;
    a->beta = split(how->beta);
    a->dbeta = how->beta;
    a->smoothing = split(how->label_smoothing);
    a->rest = split(1.0 - how->label_smoothing);
    a->dmargin = how->margin;
    a->inverse_beta = 1.0 / how->beta;
    return TT_OK;
}

tt_status fill_policy(const tt_policy* how, AnswerArgs* a) {
    if (!how || (how->level != TT_POLICY_TOKEN && how->level != TT_POLICY_SEQUENCE) || how->kl < TT_KL_1 || how->kl > TT_KL_3) return TT_ERR_ARG;
    if (!(how->clip_low >= 0.0 && how->clip_low < 1.0) || !(how->clip_high >= 0.0 && how->clip_high <= 1e6)) return TT_ERR_ARG;
    if (!(how->dual_clip == 0.0 || (how->dual_clip > 1.0 && how->dual_clip <= 1e6)) || !(how->kl_weight >= 0.0 && how->kl_weight <= 1e6)) return TT_ERR_ARG;
    if (how->level == TT_POLICY_SEQUENCE && how->per_token) return TT_ERR_ARG;
    if (a->N && !a->ref && how->kl_weight != 0.0) return TT_ERR_ARG;
    if (!aligned(how->old_dev, 4) || !aligned(how->advantages_dev, 4)) return TT_ERR_ARG;
    if ((a->N && !how->old_dev) || ((how->per_token ? a->N : a->S) && !how->advantages_dev)) return TT_ERR_ARG;
    a->old = how->old_dev;
    a->adv = how->advantages_dev;
    a->per_token = how->per_token != 0;
    a->sequence = how->level == TT_POLICY_SEQUENCE;
    a->kl = how->kl;
    a->low = (float)(1.0 - how->clip_low);
    a->high = (float)(1.0 + how->clip_high);
    a->dual = (float)how->dual_clip;
    a->tlow = split(std::log1p(-how->clip_low));
    a->thigh = split(std::log1p(how->clip_high));
    a->tdual = how->dual_clip > 0.0 ? split(std::log(how->dual_clip)) : Two{INFINITY, 0.f};
    a->kl_weight = (float)how->kl_weight;
    return TT_OK;
}

// Four values of every array at a time: all of them on 16-byte boundaries, the mask on 4.
int all_aligned(const AnswerArgs& a) {
    return aligned(a.logp, 16) && aligned(a.ref, 16) && aligned(a.mask, 4) && aligned(a.old, 16) && (!a.per_token || aligned(a.adv, 16)) &&
           aligned(a.grad, 16);
}

template <bool POLICY>
tt_status run_forward(AnswerArgs a, void* ws, size_t bytes, cudaStream_t st) {
    if (a.S == 0) return TT_OK;
    const int64_t pieces = a.S + a.chunks;
    const bool one = in_one_block(a.N, pieces);
    if (!aligned(ws, 256) || (!one && (!ws || (int64_t)bytes < pieces * kSumsBytes))) return TT_ERR_ARG;
    if (head_sms() <= 0) return TT_ERR_CUDA;
    a.part = static_cast<Sums*>(ws);
    a.vec = all_aligned(a);
    if (one) {
        k_answer_one<POLICY><<<1, kOneWarps * 32, 0, st>>>(a);
    } else {
        k_answer_sums<POLICY><<<(unsigned)((pieces + kAnswerWarps - 1) / kAnswerWarps), kAnswerWarps * 32, 0, st>>>(a);
        const int64_t out = POLICY ? (a.S + 1) / 2 : a.pairs;
        if (!launch_ahead(k_answer_finish<POLICY>, dim3((unsigned)((out + kAnswerWarps - 1) / kAnswerWarps)), kAnswerWarps * 32, 0, st, a)) return TT_ERR_CUDA;
    }
    return cudaGetLastError() == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

template <bool POLICY>
tt_status run_backward(AnswerArgs a, cudaStream_t st) {
    if (a.N == 0) return TT_OK;
    if (head_sms() <= 0) return TT_ERR_CUDA;
    a.vec = all_aligned(a);
    const int64_t pieces = a.S + 1 + a.chunks;
    k_answer_grad<POLICY><<<(unsigned)((pieces + kAnswerWarps - 1) / kAnswerWarps), kAnswerWarps * 32, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

}  // namespace
}  // namespace ttemb

using namespace ttemb;

extern "C" {

int64_t tt_emb_answers_workspace(int64_t tokens, int64_t sequences) {
    if (answer_sizes(tokens, sequences) != TT_OK) return -1;
    const int64_t pieces = sequences + (tokens > 0 ? (tokens - 1) >> piece_shift(tokens, true) : 0);
    return in_one_block(tokens, pieces) ? 0 :  // (the policy loss has the shorter pieces)
           (pieces * kSumsBytes + 255) / 256 * 256;
}

tt_status tt_emb_preference_forward(const tt_answers* answers, const tt_preference* how, float* loss_dev, float* margins_dev, float* rewards_dev,
                                    int32_t* counts_dev, int32_t* err_dev, void* ws_dev, size_t ws_bytes, tt_stream stream) {
    AnswerArgs a{};
    tt_status st = fill_answers(answers, false, &a);
    if (st == TT_OK) st = fill_preference(how, &a);
    if (st != TT_OK) return st;
    if (a.N && !a.logp) return TT_ERR_ARG;
    if (a.S && (!loss_dev || !margins_dev || !rewards_dev || !counts_dev)) return TT_ERR_ARG;
    if (!aligned(loss_dev, 4) || !aligned(margins_dev, 4) || !aligned(rewards_dev, 4) || !aligned(counts_dev, 4) || !aligned(err_dev, 4)) return TT_ERR_ARG;
    a.loss = loss_dev;
    a.margins = margins_dev;
    a.rewards = rewards_dev;
    a.counts_out = counts_dev;
    a.err = err_dev;
    return run_forward<false>(a, ws_dev, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

tt_status tt_emb_preference_backward(const tt_answers* answers, const tt_preference* how, const float* margins_dev, const int32_t* counts_dev,
                                     const float* grad_loss_dev, float* grad_logp_dev, tt_stream stream) {
    AnswerArgs a{};
    tt_status st = fill_answers(answers, false, &a);
    if (st == TT_OK) st = fill_preference(how, &a);
    if (st != TT_OK) return st;
    a.logp = a.ref = nullptr;  // not read
    if ((a.S && (!margins_dev || !counts_dev || !grad_loss_dev)) || (a.N && !grad_logp_dev)) return TT_ERR_ARG;
    if (!aligned(margins_dev, 4) || !aligned(counts_dev, 4) || !aligned(grad_loss_dev, 4) || !aligned(grad_logp_dev, 4)) return TT_ERR_ARG;
    a.margins_in = margins_dev;
    a.counts = counts_dev;
    a.grad_loss = grad_loss_dev;
    a.grad = grad_logp_dev;
    return run_backward<false>(a, reinterpret_cast<cudaStream_t>(stream));
}

tt_status tt_emb_policy_forward(const tt_answers* answers, const tt_policy* how, float* loss_dev, float* kl_dev, float* log_ratio_dev,
                                int32_t* counts_dev, int32_t* clipped_dev, int32_t* err_dev, void* ws_dev, size_t ws_bytes, tt_stream stream) {
    AnswerArgs a{};
    tt_status st = fill_answers(answers, true, &a);
    if (st == TT_OK) st = fill_policy(how, &a);
    if (st != TT_OK) return st;
    if (a.N && !a.logp) return TT_ERR_ARG;
    if (a.S && (!loss_dev || !kl_dev || !log_ratio_dev || !counts_dev || !clipped_dev)) return TT_ERR_ARG;
    if (!aligned(loss_dev, 4) || !aligned(kl_dev, 4) || !aligned(log_ratio_dev, 4) || !aligned(counts_dev, 4) || !aligned(clipped_dev, 4) ||
        !aligned(err_dev, 4))
        return TT_ERR_ARG;
    a.loss = loss_dev;
    a.kl_out = kl_dev;
    a.log_ratio = log_ratio_dev;
    a.counts_out = counts_dev;
    a.clipped = clipped_dev;
    a.err = err_dev;
    return run_forward<true>(a, ws_dev, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

tt_status tt_emb_policy_backward(const tt_answers* answers, const tt_policy* how, const float* log_ratio_dev, const int32_t* counts_dev,
                                 const float* grad_loss_dev, float* grad_logp_dev, tt_stream stream) {
    AnswerArgs a{};
    tt_status st = fill_answers(answers, true, &a);
    if (st == TT_OK) st = fill_policy(how, &a);
    if (st != TT_OK) return st;
    if (a.N && !a.logp) return TT_ERR_ARG;
    if ((a.S && (!log_ratio_dev || !counts_dev || !grad_loss_dev)) || (a.N && !grad_logp_dev)) return TT_ERR_ARG;
    if (!aligned(log_ratio_dev, 4) || !aligned(counts_dev, 4) || !aligned(grad_loss_dev, 4) || !aligned(grad_logp_dev, 4)) return TT_ERR_ARG;
    a.log_ratio_in = log_ratio_dev;
    a.counts = counts_dev;
    a.grad_loss = grad_loss_dev;
    a.grad = grad_logp_dev;
    return run_backward<true>(a, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
