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
// empty where a sequence begins there or none is).  A warp takes a piece, eight tokens a
// lane and step; pieces of one sequence are joined in their order, so results repeat.
#include <cmath>

#include "tt_units.cuh"

namespace ttemb {

constexpr int kPieceMin = 256, kPieceMax = 2048;  // tokens
constexpr int kAnswerWarps = 8;                   // pieces of a block
constexpr int kOneWarps = 32;                     // of the block that does a small call alone
constexpr int64_t kOneTokens = 8192, kOnePieces = 320;

// Sums over a piece, and over a sequence.
struct __align__(16) Sums {
    double a, b, c;  // preference: a = sum of log ratios; policy: L, k, d
    int count, clipped;
};
constexpr int64_t kSumsBytes = sizeof(Sums);
static_assert(sizeof(Sums) == 32, "layout of the workspace");

// A sum in two floats, which keeps some 48 bits: every rounding of `hi` goes to `lo` (the exact
// error of an addition: D. E. Knuth, "The Art of Computer Programming", vol. 2, 4.2.2).  Doubles
// would cost more than all else here: the device adds two a cycle and multiprocessor.
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
    __device__ __forceinline__ double value() const { return isfinite(hi) ? (double)hi + (double)lo : (double)hi; }
};

struct Threshold {  // a number in two pieces: hi + lo
    float hi, lo;
};

struct AnswerArgs {
    const float* logp;
    const float* ref;
    const uint8_t* mask;
    const int64_t* off;
    int64_t N, S, len;  // len: tokens of a sequence without offsets
    int K;
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
    float beta, smoothing, margin;
    double dbeta, dmargin;
    float* margins;
    float* rewards;
    const float* margins_in;
    // policy
    const float* old;
    const float* adv;
    int per_token, sequence, kl;
    float low, high, dual;        // 1 - clip_low, 1 + clip_high, dual_clip
    Threshold tlow, thigh, tdual;  // their logarithms
    float kl_weight;
    float* kl_out;
    float* log_ratio;
    int* clipped;
    const float* log_ratio_in;
};

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
    if (!a.off) return a.len ? t / a.len : a.S;
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
        p.e = min(p.e, (p.b / a.K + 1) * a.K);
    } else {
        p.b = (u - seqs + 1) * a.K;
        p.s = sequence_of(a, p.b);
        p.e = p.s < a.S ? offset_at(a, p.s + 1) : (with_rest ? a.N : p.b);
        p.e = min(p.e, p.b + a.K);
        if (offset_at(a, p.s) >= p.b) p.e = p.b;  // begins there: has a piece of its own
    }
    return p;
}

// x against t for x = p - q without the rounding of the difference: -1, 0, 1.
__device__ __noinline__ int side_of(float p, float q, Threshold t) {
    const double x = (double)p - (double)q, y = (double)t.hi + (double)t.lo;
    return x > y ? 1 : (x < y ? -1 : 0);
}

// exp(y) - 1 - y.  Where the three nearly cancel, its Taylor series (|y| <= 1: the first term
// left out is below 2^-28 of the sum).
__device__ __forceinline__ float exp_less_line(float y) {
    if (fabsf(y) > 1.f) return y > 64.f ? expf(y) : expf(y) - 1.f - y;  // (infinite, not inf - inf)
    float s = 1.f / 479001600.f;
    s = fmaf(s, y, 1.f / 39916800.f);
    s = fmaf(s, y, 1.f / 3628800.f);
    s = fmaf(s, y, 1.f / 362880.f);
    s = fmaf(s, y, 1.f / 40320.f);
    s = fmaf(s, y, 1.f / 5040.f);
    s = fmaf(s, y, 1.f / 720.f);
    s = fmaf(s, y, 1.f / 120.f);
    s = fmaf(s, y, 1.f / 24.f);
    s = fmaf(s, y, 1.f / 6.f);
    s = fmaf(s, y, 0.5f);
    return s * y * y;
}

// The clipped term of one token, d = p - q rounded: whether its ratio is beyond the bound, L, and dL/dx.
// The rounded d decides which side of a border x is on unless it is the rounded border itself.
struct Clipped {
    bool over;
    float term, slope;
};
__device__ __forceinline__ Clipped clip_term(const AnswerArgs& a, float adv, float d, float p, float q) {
    bool high = d > a.thigh.hi, low = d < a.tlow.hi, dual = d > a.tdual.hi;
    if (d == a.thigh.hi || d == a.tlow.hi || d == a.tdual.hi) {
        high = side_of(p, q, a.thigh) > 0;
        low = side_of(p, q, a.tlow) < 0;
        dual = side_of(p, q, a.tdual) > 0;
    }
    Clipped c;
    c.over = adv > 0.f ? high : (adv < 0.f && (low || dual));
    const float bound = adv > 0.f ? a.high : (low ? a.low : a.dual), r = expf(d);
    c.term = -adv * (c.over ? bound : r);
    c.slope = c.over ? 0.f : c.term;
    return c;
}

// k and dk/dlogp of y = reference - logp.
__device__ __forceinline__ float kl_of(const AnswerArgs& a, float y) {
    return a.kl == TT_KL_1 ? -y : (a.kl == TT_KL_2 ? 0.5f * y * y : exp_less_line(y));
}
__device__ __forceinline__ float kl_slope(const AnswerArgs& a, float y) {
    if (a.kl != TT_KL_3) return a.kl == TT_KL_1 ? 1.f : -y;
    return fabsf(y) > 1.f ? 1.f - expf(y) : -(exp_less_line(y) + y);  // 1 - exp(y)
}

// Four tokens of a piece, the first a multiple of 4.  A piece's tokens are counted from the last
// multiple of 4 before it, so that all but its first and last four are loaded whole.
struct Four {
    float lp[4], rf[4], od[4], ad[4];
    unsigned keep;  // bit 8 j + 7: token j is in the piece and counts
};
struct Span {
    int64_t first;  // a multiple of 4
    int b, e, lim;  // the piece, and the end of the arrays, from there
    __device__ __forceinline__ explicit Span(const AnswerArgs& a, const Piece& p) {
        first = p.b & ~3ll;
        b = (int)(p.b - first);
        e = (int)(p.e - first);
        lim = (int)min(a.N - first, (int64_t)1 << 20);
    }
};
__device__ __forceinline__ void load_four(const AnswerArgs& a, const Span& s, int at, bool lp, bool rf, bool od, bool ad, Four& f) {
    f.keep = 0;
    if (at >= s.e) return;
    const int64_t i = s.first + at;
    unsigned m = 0x01010101u;
    if (a.vec && at + 4 <= s.lim) {
        auto get = [&](const float* p, float (&v)[4]) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(p + i));
            v[0] = x.x;
            v[1] = x.y;
            v[2] = x.z;
            v[3] = x.w;
        };
        if (lp) get(a.logp, f.lp);
        if (rf) get(a.ref, f.rf);
        if (od) get(a.old, f.od);
        if (ad) get(a.adv, f.ad);
        if (a.mask) m = __ldg(reinterpret_cast<const unsigned*>(a.mask + i));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (at + j >= s.lim) break;
            if (lp) f.lp[j] = __ldg(a.logp + i + j);
            if (rf) f.rf[j] = __ldg(a.ref + i + j);
            if (od) f.od[j] = __ldg(a.old + i + j);
            if (ad) f.ad[j] = __ldg(a.adv + i + j);
            if (a.mask) m = (m & ~(255u << (8 * j))) | (unsigned)__ldg(a.mask + i + j) << (8 * j);
        }
    }
    f.keep = (((m & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) | m) & 0x80808080u;  // bytes that are not 0
    if (at < s.b) f.keep &= 0x80808080u << (8 * (s.b - at));
    if (at + 4 > s.e) f.keep &= 0x80808080u >> (8 * (at + 4 - s.e));
}
__device__ __forceinline__ bool kept(const Four& f, int j) { return f.keep & (0x80u << (8 * j)); }

template <bool POLICY>
__device__ Sums sum_piece(const AnswerArgs& a, const Piece& p) {
    const int lane = threadIdx.x & 31;
    Sums s{0., 0., 0., 0, 0};
    Long la, lb, lc;
    if (p.b < p.e) {
        const bool ref = a.ref != nullptr, per_token = POLICY && a.per_token, clip = POLICY && !a.sequence;
        const float seq_adv = POLICY && !a.per_token ? __ldg(a.adv + p.s) : 0.f;
        const Span span(a, p);
        for (int base = lane * 4; base - lane * 4 < span.e; base += 256) {
            Four f[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) load_four(a, span, base + h * 128, true, ref, POLICY, per_token, f[h]);
            float fa = 0.f, fb = 0.f, fc = 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                s.count += __popc(f[h].keep);
                if constexpr (!POLICY) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) fa += kept(f[h], j) ? (ref ? f[h].lp[j] - f[h].rf[j] : f[h].lp[j]) : 0.f;
                } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) fc += kept(f[h], j) ? f[h].lp[j] - f[h].od[j] : 0.f;
                if (clip) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const Clipped c = clip_term(a, per_token ? f[h].ad[j] : seq_adv, f[h].lp[j] - f[h].od[j], f[h].lp[j], f[h].od[j]);
                        fa += kept(f[h], j) ? c.term : 0.f;
                        s.clipped += kept(f[h], j) && c.over;
                    }
                }
                if (ref) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float k = kl_of(a, f[h].rf[j] - f[h].lp[j]);
                        fb += kept(f[h], j) ? k : 0.f;
                    }
                }
                }
            }
            la.add(fa);
            if (POLICY) {
                lb.add(fb);
                lc.add(fc);
            }
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        la.add_lanes(o);
        if (POLICY) {
            lb.add_lanes(o);
            lc.add_lanes(o);
        }
    }
    s.a = la.value();
    s.b = lb.value();
    s.c = lc.value();
    s.count = __reduce_add_sync(0xffffffffu, s.count);
    if (POLICY) s.clipped = __reduce_add_sync(0xffffffffu, s.clipped);
    return s;
}

// All pieces of COUNT sequences (s, s + apart ..), by a warp; lane 0 has the result.
template <int COUNT>
__device__ __forceinline__ void sum_sequences(const AnswerArgs& a, const Sums* part, int64_t s, int64_t apart, Sums (&t)[COUNT]) {
    const int lane = threadIdx.x & 31;
    int64_t b[COUNT], e[COUNT];
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
        b[i] = offset_at(a, s + i * apart);
        e[i] = offset_at(a, s + i * apart + 1);
    }
    bool one = true;
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
        const int64_t c0 = b[i] / a.K, c1 = e[i] > b[i] ? (e[i] - 1) / a.K : c0;
        t[i] = Sums{0., 0., 0., 0, 0};
        for (int64_t c = c0 + lane; c <= c1; c += 32) {  // the piece of the sequence in [c K, (c + 1) K)
            const Sums x = part[c == c0 ? s + i * apart : a.S + c - 1];
            t[i].a += x.a;
            t[i].b += x.b;
            t[i].c += x.c;
            t[i].count += x.count;
            t[i].clipped += x.clipped;
        }
        one = one && c1 == c0;
    }
    if (one) return;  // lane 0 has them whole, which is the lane that is asked
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            t[i].a += __shfl_xor_sync(0xffffffffu, t[i].a, o);
            t[i].b += __shfl_xor_sync(0xffffffffu, t[i].b, o);
            t[i].c += __shfl_xor_sync(0xffffffffu, t[i].c, o);
        }
        t[i].count = __reduce_add_sync(0xffffffffu, t[i].count);
        t[i].clipped = __reduce_add_sync(0xffffffffu, t[i].clipped);
    }
}

// dloss/dh of a pair.
__device__ __forceinline__ float pref_slope(const AnswerArgs& a, float h) {
    if (a.kind == TT_PREF_HINGE) return h < 1.f ? -1.f : 0.f;
    if (a.kind == TT_PREF_SQUARED) return 2.f * ((h - 0.5f) / a.beta) / a.beta;
    return a.smoothing / (1.f + expf(-h)) - (1.f - a.smoothing) / (1.f + expf(h));
}

// The numbers of pair u (preference) or sequence u (policy), by a warp.
template <bool POLICY>
__device__ void finish_one(const AnswerArgs& a, const Sums* part, int64_t u) {
    const bool lead = (threadIdx.x & 31) == 0;
    if (POLICY) {
        Sums one[1];
        sum_sequences<1>(a, part, u, 0, one);
        const Sums& t = one[0];
        if (!lead) return;
        const double n = t.count > 0 ? (double)t.count : 1.0, share = a.average ? 1.0 / n : 1.0;
        const float x = (float)(t.c / n);
        double term = t.a;
        int over = t.clipped;
        if (a.sequence) {
            const Clipped c = clip_term(a, a.adv[u], x, x, 0.f);
            term = t.count > 0 ? (double)c.term * t.count : 0.0;
            over = c.over ? t.count : 0;
        }
        const double k = share * t.b;
        a.log_ratio[u] = x;
        a.kl_out[u] = (float)k;
        a.loss[u] = (float)(share * term + (a.kl_weight != 0.f ? a.kl_weight * k : 0.0));
        a.counts_out[u] = t.count;
        a.clipped[u] = over;
    } else {
        Sums two[2];
        sum_sequences<2>(a, part, u, a.pairs, two);
        const Sums &c = two[0], &r = two[1];
        if (!lead) return;
        const double rc = a.dbeta * c.a / (a.average && c.count > 0 ? c.count : 1), rr = a.dbeta * r.a / (a.average && r.count > 0 ? r.count : 1);
        const float h = (float)(rc - rr - a.dmargin);
        float loss;
        if (a.kind == TT_PREF_SIGMOID) {
            const float soft = log1pf(expf(-fabsf(h)));  // log sigma(h) = min(h, 0) - soft
            loss = (1.f - a.smoothing) * (soft - fminf(h, 0.f));
            if (a.smoothing != 0.f) loss += a.smoothing * (soft + fmaxf(h, 0.f));
            if (isnan(h)) loss = h;
        } else if (a.kind == TT_PREF_HINGE) {
            loss = isnan(h) ? h : fmaxf(1.f - h, 0.f);
        } else {
            const float v = (h - 0.5f) / a.beta;
            loss = v * v;
        }
        a.loss[u] = loss;
        a.margins[u] = h;
        a.rewards[u] = (float)rc;
        a.rewards[a.pairs + u] = (float)rr;
        a.counts_out[u] = c.count;
        a.counts_out[a.pairs + u] = r.count;
    }
}

__device__ __forceinline__ void check_offsets(const AnswerArgs& a, int64_t u) {  // by one lane, u < S
    if (!a.off || !a.err) return;
    const int64_t b = a.off[u], e = a.off[u + 1];
    if (b < 0 || e < b || e > a.N || e - b > 0x7FFFFFFF || (u == 0 && b != 0)) atomicOr(a.err, kErrOffsets);
}

template <bool POLICY>
__global__ void __launch_bounds__(kAnswerWarps * 32) k_answer_sums(const __grid_constant__ AnswerArgs a) {
    const int64_t u = (int64_t)blockIdx.x * kAnswerWarps + (threadIdx.x >> 5);
    pdl_launch_dependents();
    if (u >= a.S + a.chunks) return;
    const Sums s = sum_piece<POLICY>(a, piece_of(a, u, false));
    if ((threadIdx.x & 31) == 0) {
        a.part[u] = s;
        if (u < a.S) check_offsets(a, u);
    }
}

template <bool POLICY>
__global__ void __launch_bounds__(kAnswerWarps * 32) k_answer_finish(const __grid_constant__ AnswerArgs a) {
    const int64_t u = (int64_t)blockIdx.x * kAnswerWarps + (threadIdx.x >> 5);
    pdl_wait();
    if (u < (POLICY ? a.S : a.pairs)) finish_one<POLICY>(a, a.part, u);
}

// A small call: both steps in one block.
template <bool POLICY>
__global__ void __launch_bounds__(kOneWarps * 32) k_answer_one(const __grid_constant__ AnswerArgs a) {
    __shared__ Sums part[kOnePieces];
    const int warp = threadIdx.x >> 5;
    for (int64_t u = warp; u < a.S + a.chunks; u += kOneWarps) {
        const Sums s = sum_piece<POLICY>(a, piece_of(a, u, false));
        if ((threadIdx.x & 31) == 0) {
            part[u] = s;
            if (u < a.S) check_offsets(a, u);
        }
    }
    __syncthreads();
    for (int64_t u = warp; u < (POLICY ? a.S : a.pairs); u += kOneWarps) finish_one<POLICY>(a, part, u);
}

template <bool POLICY>
__global__ void __launch_bounds__(kAnswerWarps * 32) k_answer_grad(const __grid_constant__ AnswerArgs a) {
    const int64_t u = (int64_t)blockIdx.x * kAnswerWarps + (threadIdx.x >> 5);
    if (u >= a.S + 1 + a.chunks) return;
    const int lane = threadIdx.x & 31;
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
                seq_slope = clip_term(a, adv, x, x, 0.f).slope;
            }
        } else {
            const bool chosen = p.s < a.pairs;
            const int64_t pair = chosen ? p.s : p.s - a.pairs;
            g = a.grad_loss[pair] * pref_slope(a, a.margins_in[pair]) * a.beta / (float)n;
            if (!chosen) g = -g;
        }
    }
    const bool kl = POLICY && in && a.ref && a.kl_weight != 0.f, ratio = POLICY && in && !a.sequence;
    const bool per_token = ratio && a.per_token;
    const Span span(a, p);
    for (int base = lane * 4; base - lane * 4 < span.e; base += 256) {
        Four f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            load_four(a, span, base + h * 128, kl || ratio, kl, ratio, per_token, f[h]);
            if (!in) f[h].keep = 0;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = base + h * 128;
            if (at >= span.e) continue;
            float v[4];
            if (POLICY) {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = seq_slope;
                if (ratio) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[j] = clip_term(a, per_token ? f[h].ad[j] : adv, f[h].lp[j] - f[h].od[j], f[h].lp[j], f[h].od[j]).slope;
                }
                if (kl) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] = fmaf(a.kl_weight, kl_slope(a, f[h].rf[j] - f[h].lp[j]), v[j]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = kept(f[h], j) ? g * v[j] : 0.f;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = kept(f[h], j) ? g : 0.f;
            }
            float* to = a.grad + span.first + at;
            if (a.vec && at >= span.b && at + 4 <= span.e) {
                *reinterpret_cast<float4*>(to) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (at + j >= span.b && at + j < span.e) to[j] = v[j];
            }
        }
    }
}

namespace {

tt_status answer_sizes(int64_t tokens, int64_t sequences) {
    return tokens < 0 || sequences < 0 || tokens > TT_ANSWERS_MAX_TOKENS || sequences > TT_ANSWERS_MAX_SEQUENCES ? TT_ERR_SHAPE : TT_OK;
}

// Tokens of a piece: short ones while there are few for the device, to spread; long ones cost
// fewer sums to write and join.
int piece_tokens(int64_t tokens) {
    int k = kPieceMin;
    while (k < kPieceMax && tokens / k > 8192) k *= 2;
    return k;
}

tt_status fill_answers(const tt_answers* in, AnswerArgs* a) {
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
    a->K = piece_tokens(in->tokens);
    a->chunks = in->tokens > 0 ? (in->tokens - 1) / a->K : 0;
    a->average = in->average != 0;
    if (!a->off && a->len > 0x7FFFFFFF) return TT_ERR_SHAPE;  // counts are int32
    return TT_OK;
}

tt_status fill_preference(const tt_preference* how, AnswerArgs* a) {
    if (!how || how->kind < TT_PREF_SIGMOID || how->kind > TT_PREF_SQUARED) return TT_ERR_ARG;
    if (!(how->beta > 0.0 && how->beta <= 1e6) || !(how->label_smoothing >= 0.0 && how->label_smoothing < 1.0) || !std::isfinite(how->margin))
        return TT_ERR_ARG;
    if (how->kind != TT_PREF_SIGMOID && how->label_smoothing != 0.0) return TT_ERR_ARG;
    if (a->S % 2) return TT_ERR_SHAPE;
    a->kind = how->kind;
    a->pairs = a->S / 2;
    a->beta = (float)how->beta;
    a->dbeta = how->beta;
    a->smoothing = (float)how->label_smoothing;
    a->margin = (float)how->margin;
    a->dmargin = how->margin;
    return TT_OK;
}

Threshold split(double x) {
    const float hi = (float)x;
    return {hi, (float)(x - hi)};
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
    a->tdual = how->dual_clip > 0.0 ? split(std::log(how->dual_clip)) : Threshold{INFINITY, 0.f};
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
    if ((int64_t)bytes < pieces * kSumsBytes || !ws || !aligned(ws, 256)) return TT_ERR_ARG;
    if (head_sms() <= 0) return TT_ERR_CUDA;
    a.part = static_cast<Sums*>(ws);
    a.vec = all_aligned(a);
    // one launch while a single block's reading costs less than a second launch
    if (a.N <= kOneTokens && pieces <= kOnePieces) {
        k_answer_one<POLICY><<<1, kOneWarps * 32, 0, st>>>(a);
    } else {
        k_answer_sums<POLICY><<<(unsigned)((pieces + kAnswerWarps - 1) / kAnswerWarps), kAnswerWarps * 32, 0, st>>>(a);
        const int64_t out = POLICY ? a.S : a.pairs;
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
    const int64_t pieces = sequences + (tokens > 0 ? (tokens - 1) / piece_tokens(tokens) : 0);
    return (pieces * kSumsBytes + 255) / 256 * 256;
}

tt_status tt_emb_preference_forward(const tt_answers* answers, const tt_preference* how, float* loss_dev, float* margins_dev, float* rewards_dev,
                                    int32_t* counts_dev, int32_t* err_dev, void* ws_dev, size_t ws_bytes, tt_stream stream) {
    AnswerArgs a{};
    tt_status st = fill_answers(answers, &a);
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
    tt_status st = fill_answers(answers, &a);
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
    tt_status st = fill_answers(answers, &a);
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
    tt_status st = fill_answers(answers, &a);
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
