// tt_lookup.cu -- rows of a dense table by id, times a scale, and the table's gradient.
//
// Forward: a copy with a multiplication, 8 bytes of id and 2 D elements of traffic a row.
//
// Backward: dweight[v] = scale * sum of the rows of grad_out whose id is v.  The dense gradient
// is written whole, so N D elements are read and V D written.  Positions are sorted by
// id (stable, so that a row's sum has one order), and the sorted positions are cut into
// chunks of R: the threads of a chunk, one 16-byte unit of columns each, add up its rows in
// fp32 registers, eight loads in flight whatever the ids are, and write a row where
// the id changes.  Chunks are equal work however popular an id is; what an id has in several
// chunks goes through fp32 partial sums, joined in order.  Rows that no id names are written
// with zeros by blocks that find their range of the sorted ids by bisection.
//
// The sort is a radix sort by counting (digits of up to 11 bits): per chunk of kSortChunk
// positions a histogram, scanned over the chunks of a digit by a warp, and a scatter by ranks
// within the chunk (votes per warp).  The scatter counts the next digit's histogram.
//
// Few lookups are not sorted: a block per lookup and column slice looks through all ids,
// leaves if an earlier lookup has the same, and else sums those that have it.
//
// Measured: 16,384 of 131,072 x 4096 bf16, forward: 40 us (269 MB, 6.7 TB/s).  65,521 of 50,001 x 2048 bf16: 160 us both
// ways (947 MB, 5.9 TB/s), of which the sort's three launches, which keep few multiprocessors busy, some 19.  10,240 of 1,000,000 x 64
// fp32: 54 us both ways, where the 256 MB of zeros alone need 38.  8 of 120 x 8: 5.5 us both ways.
#include <algorithm>

#include "tt_units.cuh"

namespace ttemb {

constexpr int kLkThreads = 256;
constexpr int kLkRows = 4;             // rows of a thread in the forward pass
// Lookups that are not sorted.  Each of their blocks looks through all ids, a block for 64 units of columns, so the limit lies
// lower for wide rows.  bf16 gradients of 50,001 rows, us, this way and sorted: 64 wide, 300 lookups 6 and 15, 1,024 10 and 17, 2,048 20 and
// 20; 2048 wide, 300 39 and 40, 600 46 and 41, 1,024 56 and 41 (added to a gradient: 9 and 18, 16 and 18, 26 and 19).
constexpr int kSmallRows = 1024;
constexpr int kSortChunk = 2048;
constexpr int kSortBlock = 512;
constexpr int kSortW = kSortBlock / 32;
// Up to so many chunks a scatter sums the histograms itself.  Gradients of 50,001 x 256, us, so and by a launch of its own: 2 chunks 22 and
// 25, 8 chunks 27 and 27, 16 chunks 34 and 30, 32 chunks 39 and 36, 64 chunks 52 and 42.
constexpr int kFoldChunks = 32;
constexpr int kDigitBits = 11;
constexpr int kMaxPasses = 3;
constexpr int kZeroRows = 2048;        // most table rows of a block that writes zeros
constexpr int64_t kSmallTable = 1 << 20;  // bytes: a table that few lookups' own launch clears (beyond, a launch ahead of it, 16 bytes at a time)
constexpr int kChunkSlots = 4096;      // sorted positions staged by a block
constexpr int kInFlight = 8;

struct LookupArgs {
    const void* in;   // weight (forward) or grad_out
    int64_t in_ld;
    void* out;        // out or grad_weight
    int64_t out_ld;
    const int64_t* ids;
    int64_t N, V, pad;
    int units;        // of a row
    int D;
    int lanes;        // threads of a row (a power of two, at most kLkThreads)
    float scale;
    int accumulate;
    int* err;
    // backward, sorted
    int R;            // sorted positions of a chunk
    int64_t chunks;
    int64_t sum_blocks;  // then blocks that write zeros
    int zero_rows;       // table rows of one of these
    int64_t zero_first;  // the first row that the sort's launches have left to them
    int slices;          // column slices of `lanes` units
    const uint32_t* keys;  // [m] sorted ids
    const uint32_t* pos;   // [m] their positions
    const int* m;
    float* head;           // [chunks][D] sum of a chunk's first id where it began before the chunk
    float* tail;           // [chunks][D] of its last id where that began in the chunk and goes on
};

template <class T, int VEC>
__global__ void __launch_bounds__(kLkThreads) k_lookup(const __grid_constant__ LookupArgs a) {
    const int lane = threadIdx.x & (a.lanes - 1), sub = threadIdx.x / a.lanes, per = kLkThreads / a.lanes;
    const int64_t n0 = (int64_t)blockIdx.x * per * kLkRows + sub;
    const int u = blockIdx.y * a.lanes + lane;
    if (u >= a.units) return;
    int64_t id[kLkRows];
#pragma unroll
    for (int i = 0; i < kLkRows; ++i) {
        const int64_t n = n0 + (int64_t)i * per;
        id[i] = n < a.N ? __ldg(a.ids + n) : 0;
    }
    Raw<T, VEC> r[kLkRows];
#pragma unroll
    for (int i = 0; i < kLkRows; ++i) {
        const int64_t n = n0 + (int64_t)i * per;
        const bool ok = id[i] >= 0 && id[i] < a.V;
        r[i] = raw_zero<T, VEC>();
        if (ok && n < a.N) r[i] = __ldg(unit_at<T, VEC>(static_cast<const T*>(a.in), id[i], a.in_ld, u));
        if (!ok && u == 0 && a.err) atomicOr(a.err, kErrIndex);
        if (!ok) id[i] = -1;
    }
#pragma unroll
    for (int i = 0; i < kLkRows; ++i) {
        const int64_t n = n0 + (int64_t)i * per;
        if (n >= a.N) break;
        float v[VEC];
        unpack<T, VEC>(r[i], v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = id[i] >= 0 ? v[j] * a.scale : 0.f;
        *unit_at<T, VEC>(static_cast<T*>(a.out), n, a.out_ld, u) = pack<T, VEC>(v);
    }
}

// ---------------------------------------------------------------- sort by id

// Rows of the gradient that a launch of the sort writes with zeros beside its own work: the sort is a chain of short
// launches that leave most of the device idle, and zeros need no sorted ids.  Rows that are named are
// written again by the sums.
struct ZeroRows {
    uint8_t* out;
    int64_t row_bytes, pitch;  // of a row, and from row to row
    int64_t rows;              // [0, rows)
};
__device__ void write_zeros(const ZeroRows& z, int block, int blocks) {
    const int64_t thread = (int64_t)block * blockDim.x + threadIdx.x, threads = (int64_t)blocks * blockDim.x;
    auto clear = [](uint8_t* p, int64_t bytes, int64_t first, int64_t step) {  // 16 bytes at a time, and what is left at both ends
        const int64_t head = min(bytes, (int64_t)(-(intptr_t)p & 15)), n = (bytes - head) / 16;
        uint4* q = reinterpret_cast<uint4*>(p + head);
#pragma unroll 8
        for (int64_t i = first; i < n; i += step) q[i] = make_uint4(0, 0, 0, 0);
        const int64_t tail = head + n * 16;
        if (first * 2 < head) reinterpret_cast<uint16_t*>(p)[first] = 0;
        if (first * 2 < bytes - tail) reinterpret_cast<uint16_t*>(p + tail)[first] = 0;
    };
    if (z.row_bytes == z.pitch || z.rows == 1) {
        if (z.rows > 0) clear(z.out, z.rows * z.row_bytes, thread, threads);
        return;
    }
    const int warps = blockDim.x / 32;
    for (int64_t r = (int64_t)block * warps + (threadIdx.x >> 5); r < z.rows; r += (int64_t)blocks * warps)
        clear(z.out + r * z.pitch, z.row_bytes, threadIdx.x & 31, 32);
}
__global__ void __launch_bounds__(512) k_lookup_zero(const __grid_constant__ ZeroRows z) {
    pdl_launch_dependents();
    write_zeros(z, blockIdx.x, gridDim.x);
}

struct SortArgs {
    const int64_t* ids;
    int64_t N, V, pad;
    int nch, passes, bits[kMaxPasses], bins[kMaxPasses];
    int* H[kMaxPasses];      // [nch][bins], after its scan the sum over earlier chunks
    int* total[kMaxPasses];  // [bins]
    uint32_t* keys[2];
    uint32_t* pos[2];
    int* m;                  // ids that count
    int* err;
};

__device__ __forceinline__ int64_t key_of(const SortArgs& a, int64_t id) {  // -1: does not count
    return id < 0 || id >= a.V || id == a.pad ? -1 : id;
}

__global__ void __launch_bounds__(kSortBlock) k_lookup_hist(const __grid_constant__ SortArgs a, const __grid_constant__ ZeroRows z) {
    extern __shared__ int bins_s[];
    const int c = blockIdx.x;
    pdl_launch_dependents();
    if (c >= a.nch) {
        write_zeros(z, c - a.nch, gridDim.x - a.nch);
        return;
    }
    const int64_t lo = (int64_t)c * kSortChunk;
    int64_t id[kSortChunk / kSortBlock];
#pragma unroll
    for (int i = 0; i < kSortChunk / kSortBlock; ++i) {
        const int64_t n = lo + i * kSortBlock + threadIdx.x;
        id[i] = n < a.N ? a.ids[n] : a.pad;
    }
    for (int i = threadIdx.x; i < a.bins[0]; i += kSortBlock) bins_s[i] = 0;
    for (int p = 1; p < a.passes; ++p)  // counted by the scatter before
        for (int64_t i = (int64_t)c * kSortBlock + threadIdx.x; i < (int64_t)a.bins[p] * a.nch; i += (int64_t)a.nch * kSortBlock) a.H[p][i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSortChunk / kSortBlock; ++i) {
        const int64_t n = lo + i * kSortBlock + threadIdx.x;
        if (n >= a.N) break;
        const int64_t k = key_of(a, id[i]);
        if (k >= 0)
            atomicAdd(&bins_s[(int)k & (a.bins[0] - 1)], 1);
        else if (a.err && (id[i] < 0 || id[i] >= a.V))
            atomicOr(a.err, kErrIndex);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.bins[0]; i += kSortBlock) a.H[0][(int64_t)c * a.bins[0] + i] = bins_s[i];
}

// Sums over earlier chunks, and over all, of 32 digits: a digit to a lane, equal runs of chunks to the warps.
__global__ void __launch_bounds__(kSortBlock) k_lookup_scan(const __grid_constant__ SortArgs a, int p) {
    __shared__ int run_s[kSortW][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, b = blockIdx.x * 32 + lane, bins = a.bins[p];
    pdl_entry();
    const bool in = b < bins;
    const int from = (int)((int64_t)a.nch * w / kSortW), to = (int)((int64_t)a.nch * (w + 1) / kSortW);
    int* h = a.H[p] + (in ? b : 0);
    int sum = 0;
#pragma unroll 8
    for (int c = from; c < to; ++c) sum += h[(int64_t)c * bins];
    run_s[w][lane] = sum;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kSortW; ++i) {
        before += i < w ? run_s[i][lane] : 0;
        all += run_s[i][lane];
    }
    if (!in) return;
#pragma unroll 8
    for (int c = from; c < to; ++c) {
        const int v = h[(int64_t)c * bins];
        h[(int64_t)c * bins] = before;
        before += v;
    }
    if (w == 0) a.total[p][b] = all;
}

// Exclusive scan of x over the block's WARPS warps; *total: the sum.
template <int WARPS>
__device__ __forceinline__ int block_scan(int x, int* sh, int* total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    __syncthreads();
    if (lane == 31) sh[w] = s;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
        before += i < w ? sh[i] : 0;
        all += sh[i];
    }
    *total = all;
    return before + s - x;
}

__global__ void __launch_bounds__(kSortBlock) k_lookup_scatter(const __grid_constant__ SortArgs a, const __grid_constant__ ZeroRows z, int p) {
    extern __shared__ int sm[];
    __shared__ int sh[kSortW];
    const int bins = a.bins[p], c = blockIdx.x, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    pdl_launch_dependents();
    if (c >= a.nch) {
        write_zeros(z, c - a.nch, gridDim.x - a.nch);
        return;
    }
    int* base = sm;                                                // [bins]
    uint16_t* cnt = reinterpret_cast<uint16_t*>(sm + bins);        // [kSortW][bins], at most kSortChunk each
    uint32_t* cnt2 = reinterpret_cast<uint32_t*>(cnt);             // two bins at a time
    for (int i = threadIdx.x; i < kSortW * bins / 2; i += kSortBlock) cnt2[i] = 0;
    int shift = 0;
    for (int i = 0; i < p; ++i) shift += a.bits[i];
    const int64_t lo = (int64_t)c * kSortChunk;
    // a warp's positions are consecutive: 4 x 32
    constexpr int kPer = kSortChunk / kSortBlock;
    uint32_t key[kPer], at[kPer];
    int digit[kPer], rank[kPer];
    uint16_t* mine = cnt + w * bins;
    const int64_t first = lo + w * (kSortChunk / kSortW);
    if (p == 0) {  // the ids need no wait
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int64_t n = first + i * 32 + lane, k = n < a.N ? key_of(a, a.ids[n]) : -1;
            key[i] = (uint32_t)k;
            at[i] = (uint32_t)n;
            digit[i] = k >= 0 ? (int)k & (bins - 1) : -1;
        }
    }
    pdl_wait();
    if (p > 0) {
        const int64_t count = *a.m;
        if (lo >= count) return;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int64_t n = first + i * 32 + lane;
            digit[i] = -1;
            key[i] = at[i] = 0;
            if (n < count) {
                key[i] = a.keys[(p - 1) & 1][n];
                at[i] = a.pos[(p - 1) & 1][n];
                digit[i] = (int)(key[i] >> shift) & (bins - 1);
            }
        }
    }
    // where the digits begin: consecutive ones to a thread
    constexpr int kMost = (1 << kDigitBits) / kSortBlock;
    const int each = (bins + kSortBlock - 1) / kSortBlock;
    int begin[kMost], sum = 0;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        const int b = threadIdx.x * each + i;
        int all = 0, before = 0;
        if (i < each && b < bins) {
            const int* h = a.H[p] + b;
            if (a.nch <= kFoldChunks) {
#pragma unroll 32
                for (int k = 0; k < a.nch; ++k) {
                    const int v = h[k * bins];
                    all += v;
                    before += k < c ? v : 0;
                }
            } else {
                all = a.total[p][b];
                before = h[(int64_t)c * bins];
            }
        }
        begin[i] = sum + before;
        sum += all;
    }
    int carry;
    const int thread_begin = block_scan<kSortW>(sum, sh, &carry);
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        const int b = threadIdx.x * each + i;
        if (i < each && b < bins) base[b] = thread_begin + begin[i];
    }
    if (p == 0 && c == 0 && threadIdx.x == 0) *a.m = carry;
    unsigned peers[kPer];  // lanes with the same digit
#pragma unroll
    for (int i = 0; i < kPer; ++i) peers[i] = __ballot_sync(0xffffffffu, digit[i] >= 0);
    for (int bit = 1; bit < bins; bit *= 2) {  // a vote for each bit costs a fraction of a match
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const unsigned with = __ballot_sync(0xffffffffu, digit[i] & bit);
            peers[i] &= digit[i] & bit ? with : ~with;
        }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const unsigned m = peers[i];
        const int leader = digit[i] >= 0 ? __ffs(m) - 1 : lane;
        int before = 0;
        if (digit[i] >= 0 && lane == leader) {
            before = mine[digit[i]];
            mine[digit[i]] = (uint16_t)(before + __popc(m));
        }
        rank[i] = __shfl_sync(0xffffffffu, before, leader) + __popc(m & lanemask_lt());
        __syncwarp();
    }
    __syncthreads();
    for (int b = threadIdx.x; b < bins / 2; b += kSortBlock) {  // sums over earlier warps: no carry from bin to bin
        uint32_t run = 0;
#pragma unroll
        for (int i = 0; i < kSortW; ++i) {
            const uint32_t v = cnt2[i * (bins / 2) + b];
            cnt2[i * (bins / 2) + b] = run;
            run += v;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const bool in = digit[i] >= 0;
        const int to = in ? base[digit[i]] + mine[digit[i]] + rank[i] : 0;
        if (in) {
            a.keys[p & 1][to] = key[i];
            a.pos[p & 1][to] = at[i];
        }
        if (p + 1 < a.passes) {
            // one addition for a popular id's lookups: those that go to one count with the digit's first
            const int64_t next = (int64_t)(to / kSortChunk) * a.bins[p + 1] + ((key[i] >> (shift + a.bits[p])) & (a.bins[p + 1] - 1));
            const int leader = in ? __ffs(peers[i]) - 1 : lane;
            const bool follows = __shfl_sync(0xffffffffu, (int)next, leader) == (int)next;
            const unsigned same = __ballot_sync(0xffffffffu, follows) & peers[i];
            if (in && (lane == leader || !follows)) atomicAdd(&a.H[p + 1][next], lane == leader ? __popc(same) : 1);
        }
    }
}

// ---------------------------------------------------------------- sums

// A unit of a row of partial sums.
template <int VEC>
__device__ __forceinline__ void put_part(float* to, const float (&v)[VEC]) {
    if constexpr (VEC < 4) {  // a row of an odd number of units does not begin on 16 bytes
#pragma unroll
        for (int q = 0; q < VEC; ++q) to[q] = v[q];
    } else {
#pragma unroll
        for (int q = 0; q < VEC; q += 4) *reinterpret_cast<float4*>(to + q) = make_float4(v[q], v[q + 1], v[q + 2], v[q + 3]);
    }
}
template <int VEC>
__device__ __forceinline__ void add_part(const float* from, float (&v)[VEC]) {
    if constexpr (VEC < 4) {
#pragma unroll
        for (int q = 0; q < VEC; ++q) v[q] += from[q];
    } else {
#pragma unroll
        for (int q = 0; q < VEC; q += 4) {
            const float4 x = *reinterpret_cast<const float4*>(from + q);
            v[q] += x.x;
            v[q + 1] += x.y;
            v[q + 2] += x.z;
            v[q + 3] += x.w;
        }
    }
}

// scale * v to a row of the gradient, or added to it.
template <class T, int VEC>
__device__ __forceinline__ void put_unit(const LookupArgs& a, int64_t row, int u, float (&v)[VEC]) {
    Raw<T, VEC>* p = unit_at<T, VEC>(static_cast<T*>(a.out), row, a.out_ld, u);
    if (a.accumulate) {
        float o[VEC];
        unpack<T, VEC>(*p, o);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = fmaf(v[j], a.scale, o[j]);
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] *= a.scale;
    }
    *p = pack<T, VEC>(v);
}

// The first of keys[0, m) that is not below `key`; the whole warp, 32 probes a step.
__device__ int first_not_below(const uint32_t* keys, int m, uint32_t key) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = m;  // the answer is in [lo, hi]
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const unsigned below = __ballot_sync(0xffffffffu, at < hi && keys[at] < key);
        const int n = __popc(below);  // sorted: the first n probes
        if (n == 0) return lo;
        hi = min(hi, lo + n * step);
        lo += (n - 1) * step + 1;
    }
    return lo;
}

// Rows [r0, r0 + rows) that are not flagged, with zeros.
template <class T, int VEC>
__device__ void zero_rows(const LookupArgs& a, const uint8_t* named, int64_t r0, int rows) {
    const int lane = threadIdx.x & (a.lanes - 1), sub = threadIdx.x / a.lanes, per = kLkThreads / a.lanes;
    for (int r = sub; r < rows; r += per) {
        if (named[r]) continue;
        Raw<T, VEC>* p = unit_at<T, VEC>(static_cast<T*>(a.out), r0 + r, a.out_ld, 0);
#pragma unroll 4
        for (int u = lane; u < a.units; u += a.lanes) p[u] = raw_zero<T, VEC>();
    }
}

template <class T, int VEC>
__global__ void __launch_bounds__(kLkThreads) k_lookup_sums(const __grid_constant__ LookupArgs a) {
    __shared__ uint32_t keys_s[kChunkSlots], pos_s[kChunkSlots];
    pdl_entry();
    const int m = *a.m;
    if (blockIdx.x >= a.sum_blocks) {
        uint8_t* named = reinterpret_cast<uint8_t*>(keys_s);
        int* range = reinterpret_cast<int*>(pos_s);
        const int64_t r0 = a.zero_first + (blockIdx.x - a.sum_blocks) * a.zero_rows;
        const int rows = (int)min((int64_t)a.zero_rows, a.V - r0);
        for (int r = threadIdx.x; r < rows; r += kLkThreads) named[r] = 0;
        const int w = threadIdx.x >> 5;
        if (w < 2) {
            const int at = first_not_below(a.keys, m, (uint32_t)(r0 + w * rows));
            if ((threadIdx.x & 31) == 0) range[w] = at;
        }
        __syncthreads();
        for (int i = range[0] + threadIdx.x; i < range[1]; i += kLkThreads) named[a.keys[i] - (uint32_t)r0] = 1;
        __syncthreads();
        zero_rows<T, VEC>(a, named, r0, rows);
        return;
    }
    const int lane = threadIdx.x & (a.lanes - 1), sub = threadIdx.x / a.lanes, per = kLkThreads / a.lanes;
    const int64_t block = blockIdx.x / a.slices;
    const int u = (int)(blockIdx.x - block * a.slices) * a.lanes + lane;
    const int64_t first = block * per * a.R;  // of the block's chunks
    if (first >= m) return;
    const int staged = (int)min((int64_t)per * a.R, m - first);
    for (int i = threadIdx.x; i < staged; i += kLkThreads) {
        keys_s[i] = a.keys[first + i];
        pos_s[i] = a.pos[first + i];
    }
    __syncthreads();
    const int64_t j = block * per + sub, b = j * a.R, e = min(b + a.R, (int64_t)m);
    if (b >= m || u >= a.units) return;
    const uint32_t* k = keys_s + sub * a.R;
    const uint32_t* p = pos_s + sub * a.R;
    const int n = (int)(e - b);
    const bool goes_back = b > 0 && a.keys[b - 1] == k[0], goes_on = e < m && a.keys[e] == k[n - 1];
    const T* in = static_cast<const T*>(a.in);
    float acc[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
    uint32_t cur = k[0];
    bool whole = !goes_back;  // the current id began in this chunk
    for (int t = 0; t < n; t += kInFlight) {
        Raw<T, VEC> r[kInFlight];
#pragma unroll
        for (int i = 0; i < kInFlight; ++i)
            if (t + i < n) r[i] = __ldcs(unit_at<T, VEC>(in, p[t + i], a.in_ld, u));
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            if (t + i >= n) break;
            const uint32_t key = k[t + i];
            if (key != cur) {
                if (whole) {
                    put_unit<T, VEC>(a, cur, u, acc);
                } else {
                    put_part<VEC>(a.head + j * a.D + u * VEC, acc);
                }
#pragma unroll
                for (int q = 0; q < VEC; ++q) acc[q] = 0.f;
                cur = key;
                whole = true;
            }
            float v[VEC];
            unpack<T, VEC>(r[i], v);
#pragma unroll
            for (int q = 0; q < VEC; ++q) acc[q] += v[q];
        }
    }
    if (whole && !goes_on) {
        put_unit<T, VEC>(a, cur, u, acc);
    } else {
        put_part<VEC>((whole ? a.tail : a.head) + j * a.D + u * VEC, acc);
    }
}

// The id that begins in chunk j and goes on: its partial sums, in order.  A block per chunk and slice of
// `lanes` units; where these leave threads, they take the partial sums in turn.
template <class T, int VEC>
__global__ void __launch_bounds__(kLkThreads) k_lookup_join(const __grid_constant__ LookupArgs a) {
    __shared__ float part[kLkThreads * VEC];
    const int lane = threadIdx.x & (a.lanes - 1), sub = threadIdx.x / a.lanes, per = kLkThreads / a.lanes;
    const int64_t j = blockIdx.x / a.slices;
    const int u = (int)(blockIdx.x - j * a.slices) * a.lanes + lane;
    const int64_t b = j * a.R, e = b + a.R;
    pdl_entry();
    const int64_t m = *a.m;
    if (e >= m) return;
    const uint32_t key = a.keys[e - 1], after = a.keys[e], before = b > 0 ? a.keys[b - 1] : ~0u;  // ids are below 2^30
    if (after != key || before == key) return;
    int64_t last = j + 1;  // the last chunk that has it: those whose first position has it
    for (bool more = true; more;) {
        const int64_t at = (last + 1 + (threadIdx.x & 31)) * a.R;
        const unsigned has = __ballot_sync(0xffffffffu, at < m && a.keys[at < m ? at : 0] == key);
        last += __popc(has);
        more = has == 0xffffffffu;
    }
    float s[VEC];
#pragma unroll
    for (int q = 0; q < VEC; ++q) s[q] = 0.f;
    if (u < a.units) {
        if (sub == 0) add_part<VEC>(a.tail + j * a.D + u * VEC, s);
        const float* from = a.head + (int64_t)u * VEC;
#pragma unroll 4
        for (int64_t c = j + (sub ? sub : per); c <= last; c += per) add_part<VEC>(from + c * a.D, s);
    }
    if (per > 1) {
#pragma unroll
        for (int q = 0; q < VEC; ++q) part[q * kLkThreads + threadIdx.x] = s[q];
        __syncthreads();
        if (sub > 0) return;
        for (int i = 1; i < per && j + i <= last; ++i)
#pragma unroll
            for (int q = 0; q < VEC; ++q) s[q] += part[q * kLkThreads + i * a.lanes + lane];
    }
    if (u < a.units) put_unit<T, VEC>(a, key, u, s);
}

// Few lookups: a block per lookup and slice of `lanes` units, then (small tables) blocks that write zeros.
template <class T, int VEC>
__global__ void __launch_bounds__(kLkThreads) k_lookup_few(const __grid_constant__ LookupArgs a) {
    pdl_launch_dependents();
    __shared__ int ids[kSmallRows];
    __shared__ union {
        int list[kSmallRows];
        float part[kLkThreads * VEC];
        uint8_t named[kZeroRows];
    } s;
    __shared__ int sh[kLkThreads / 32];
    const int N = (int)a.N;
    for (int n = threadIdx.x; n < N; n += kLkThreads) {
        const int64_t id = a.ids[n];
        const bool in = id >= 0 && id < a.V;
        if (!in && a.err && blockIdx.x == 0) atomicOr(a.err, kErrIndex);
        ids[n] = in && id != a.pad ? (int)id : -1;
    }
    __syncthreads();
    if (blockIdx.x >= a.sum_blocks) {
        const int64_t r0 = (blockIdx.x - a.sum_blocks) * a.zero_rows;
        const int rows = (int)min((int64_t)a.zero_rows, a.V - r0);
        for (int r = threadIdx.x; r < rows; r += kLkThreads) s.named[r] = 0;
        __syncthreads();
        for (int n = threadIdx.x; n < N; n += kLkThreads) {
            const int64_t r = (int64_t)ids[n] - r0;
            if (ids[n] >= 0 && r >= 0 && r < rows) s.named[r] = 1;
        }
        __syncthreads();
        zero_rows<T, VEC>(a, s.named, r0, rows);
        return;
    }
    const int n0 = (int)(blockIdx.x / a.slices), slice = (int)(blockIdx.x - (int64_t)n0 * a.slices);
    const int id = ids[n0];
    if (id < 0) {  // the zeros have to be there when this launch has ended, whatever the ids are
        pdl_wait();
        return;
    }
    // the lookups with this id, in order; a thread's are consecutive
    constexpr int kPer = kSmallRows / kLkThreads;
    int mine[kPer], found = 0;
    bool earlier = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int n = threadIdx.x * kPer + i;
        if (n < N && ids[n] == id) {
            earlier |= n < n0;
            mine[found++] = n;
        }
    }
    if (__syncthreads_or(earlier)) return;  // (the block of the id's first lookup waits)
    int count;
    const int at = block_scan<kLkThreads / 32>(found, sh, &count);
    for (int i = 0; i < found; ++i) s.list[at + i] = mine[i];
    __syncthreads();
    const int lane = threadIdx.x & (a.lanes - 1), sub = threadIdx.x / a.lanes, per = kLkThreads / a.lanes;
    const int u = slice * a.lanes + lane;
    const T* in = static_cast<const T*>(a.in);
    float acc[VEC];
#pragma unroll
    for (int q = 0; q < VEC; ++q) acc[q] = 0.f;
    const int b = (count * sub + per - 1) / per, e = (count * (sub + 1) + per - 1) / per;  // one lookup: the first share's
    if (u < a.units) {
        for (int t = b; t < e; t += kInFlight) {
            Raw<T, VEC> r[kInFlight];
#pragma unroll
            for (int i = 0; i < kInFlight; ++i) r[i] = t + i < e ? __ldg(unit_at<T, VEC>(in, s.list[t + i], a.in_ld, u)) : raw_zero<T, VEC>();
#pragma unroll
            for (int i = 0; i < kInFlight; ++i) {
                float v[VEC];
                unpack<T, VEC>(r[i], v);
                if (t + i < e) {
#pragma unroll
                    for (int q = 0; q < VEC; ++q) acc[q] += v[q];
                }
            }
        }
    }
    pdl_wait();  // the row may be zeros by now, and not later
    if (count > 1 && per > 1) {  // the shares in order
        __syncthreads();
#pragma unroll
        for (int q = 0; q < VEC; ++q) s.part[q * kLkThreads + threadIdx.x] = acc[q];
        __syncthreads();
        if (sub == 0)
            for (int i = 1; i < per; ++i)
#pragma unroll
                for (int q = 0; q < VEC; ++q) acc[q] += s.part[q * kLkThreads + i * a.lanes + lane];
    }
    if (sub == 0 && u < a.units) put_unit<T, VEC>(a, id, u, acc);
}

// ---------------------------------------------------------------- host

namespace {

int esize(int dtype) { return dtype == TT_F32 ? 4 : 2; }

tt_status lookup_sizes(int64_t rows, int64_t vocab, int64_t dim, int dtype) {
    if (dtype != TT_F32 && dtype != TT_BF16 && dtype != TT_F16) return TT_ERR_ARG;
    if (rows < 0 || rows > TT_LOOKUP_MAX_ROWS || vocab < 1 || vocab > TT_HEAD_MAX_VOCAB || dim < 1 || dim > TT_HEAD_MAX_DIM) return TT_ERR_SHAPE;
    return TT_OK;
}

// How a backward pass sorts and cuts its lookups; sizes only, so that the workspace's are known.
struct LookupPlan {
    bool sorted;
    int nch, passes, bits[kMaxPasses], bins[kMaxPasses], R;
    int64_t chunks;
    // the workspace's blocks
    int* H[kMaxPasses];
    int* total[kMaxPasses];
    uint32_t* keys[2];
    uint32_t* pos[2];
    int* m;
    float* head;
    float* tail;
    size_t bytes;
};

LookupPlan lookup_plan(int64_t N, int64_t V, int D, int dtype, void* ws) {
    LookupPlan p{};
    p.sorted = N > kSmallRows;
    if (!p.sorted) return p;
    int bits = 1;
    while ((1ll << bits) < V) ++bits;
    p.passes = (bits + kDigitBits - 1) / kDigitBits;
    for (int i = 0; i < p.passes; ++i) {
        p.bits[i] = (bits + p.passes - 1) / p.passes;
        p.bins[i] = 1 << p.bits[i];
    }
    p.nch = (int)((N + kSortChunk - 1) / kSortChunk);
    // long chunks leave fewer partial sums; short ones while the device would not be full
    const int64_t units = ((int64_t)D * esize(dtype) + 15) / 16;
    const int per = kLkThreads / pow2_at_least(units, kLkThreads);
    p.R = std::min(256, kChunkSlots / per);
    while (p.R > 16 && N / p.R * units < 131072) p.R /= 2;
    p.chunks = (N + p.R - 1) / p.R;
    uint8_t* base = static_cast<uint8_t*>(ws);
    size_t used = 0;
    auto get = [&](size_t n) {
        uint8_t* at = base ? base + used : nullptr;
        used += (n + 255) / 256 * 256;
        return at;
    };
    for (int i = 0; i < p.passes; ++i) {
        p.H[i] = reinterpret_cast<int*>(get((size_t)p.bins[i] * p.nch * 4));
        p.total[i] = reinterpret_cast<int*>(get((size_t)p.bins[i] * 4));
    }
    for (int i = 0; i < 2; ++i) {
        p.keys[i] = reinterpret_cast<uint32_t*>(get((size_t)N * 4));
        p.pos[i] = reinterpret_cast<uint32_t*>(get((size_t)N * 4));
    }
    p.m = reinterpret_cast<int*>(get(4));
    p.head = reinterpret_cast<float*>(get((size_t)p.chunks * D * 4));
    p.tail = reinterpret_cast<float*>(get((size_t)p.chunks * D * 4));
    p.bytes = used;
    return p;
}

void set_units(LookupArgs* a, int vec, int most) {
    a->units = a->D / vec;
    a->lanes = pow2_at_least(a->units, most);
    a->slices = (a->units + a->lanes - 1) / a->lanes;
}

template <class T, int VEC>
tt_status forward_launch(LookupArgs a, cudaStream_t st) {
    set_units(&a, VEC, kLkThreads);
    const int per = kLkThreads / a.lanes * kLkRows;
    k_lookup<T, VEC><<<dim3((unsigned)((a.N + per - 1) / per), (unsigned)a.slices), kLkThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

template <class T, int VEC>
tt_status backward_launch(LookupArgs a, const LookupPlan& p, const int64_t* ids, int sms, int dev, cudaStream_t st) {
    // some 128 KB of table rows to a block that writes zeros
    a.zero_rows = (int)std::max<int64_t>(1, std::min<int64_t>(kZeroRows, 131072 / ((int64_t)a.D * (int64_t)sizeof(T))));
    // the rows that other launches clear, in turn from the table's beginning
    const int64_t row_bytes = (int64_t)a.D * (int64_t)sizeof(T), pitch = a.out_ld * (int64_t)sizeof(T);
    const int64_t rows = a.accumulate ? 0 : a.V;
    int64_t cleared = 0;
    auto take = [&](int64_t bytes, int* blocks) {
        ZeroRows z{static_cast<uint8_t*>(a.out) + cleared * pitch, row_bytes, pitch, std::min(rows - cleared, bytes / row_bytes)};
        cleared += z.rows;
        *blocks = z.rows ? (int)std::min<int64_t>(4 * sms, (z.rows * row_bytes + 65535) / 65536) : 0;
        return z;
    };
    int extra;
    if (!p.sorted) {
        set_units(&a, VEC, 64);
        a.sum_blocks = a.N * a.slices;
        if (rows * row_bytes > kSmallTable) {
            const ZeroRows z = take(rows * row_bytes, &extra);
            k_lookup_zero<<<extra, 512, 0, st>>>(z);
            if (cudaGetLastError() != cudaSuccess) return TT_ERR_CUDA;
            if (a.N == 0) return TT_OK;
            return launch_ahead(k_lookup_few<T, VEC>, dim3((unsigned)a.sum_blocks), kLkThreads, 0, st, a) ? TT_OK : TT_ERR_CUDA;
        }
        a.zero_rows = (int)std::max<int64_t>(1, std::min<int64_t>(kZeroRows, 8192 / row_bytes));
        const int64_t blocks = a.sum_blocks + (rows + a.zero_rows - 1) / a.zero_rows;
        if (blocks == 0) return TT_OK;
        k_lookup_few<T, VEC><<<(unsigned)blocks, kLkThreads, 0, st>>>(a);  // a call's first launch waits for what ran before
        return cudaGetLastError() == cudaSuccess ? TT_OK : TT_ERR_CUDA;
    }
    SortArgs s{};
    s.ids = ids;
    s.N = a.N;
    s.V = a.V;
    s.pad = a.pad;
    s.nch = p.nch;
    s.passes = p.passes;
    for (int i = 0; i < p.passes; ++i) {
        s.bits[i] = p.bits[i];
        s.bins[i] = p.bins[i];
        s.H[i] = p.H[i];
        s.total[i] = p.total[i];
    }
    for (int i = 0; i < 2; ++i) {
        s.keys[i] = p.keys[i];
        s.pos[i] = p.pos[i];
    }
    s.m = p.m;
    s.err = a.err;
    constexpr size_t kScatterSmem = (sizeof(int) + sizeof(uint16_t) * kSortW) << kDigitBits;
    struct Tag {};
    if (!allow_smem<Tag>(k_lookup_scatter, dev, kScatterSmem)) return TT_ERR_CUDA;
    // Where few rows can be named the sort's launches write all zeros, the histogram a share and each scatter
    // two (10,240 lookups of 1,000,000 x 64 fp32, 256 MB of zeros: 62 us with a third of them there, 57 with all).  Where many can,
    // the sums do it, which leave those out (65,521 of 50,001 x 2048 bf16: 182 with half of the table there, 178 without), a row at a
    // time: not where rows are not of whole 16 bytes.
    const bool all = a.N * 4 <= a.V || VEC * sizeof(T) < 16;
    const int64_t share = all ? rows * row_bytes / (2 * p.passes + 1) + row_bytes : 0;
    const ZeroRows zh = take(share, &extra);
    k_lookup_hist<<<p.nch + extra, kSortBlock, sizeof(int) * p.bins[0], st>>>(s, zh);
    if (cudaGetLastError() != cudaSuccess) return TT_ERR_CUDA;
    for (int i = 0; i < p.passes; ++i) {
        if (p.nch > kFoldChunks && !launch_ahead(k_lookup_scan, dim3((p.bins[i] + 31) / 32), kSortBlock, 0, st, s, i)) return TT_ERR_CUDA;
        const ZeroRows zs = take(all && i + 1 == p.passes ? rows * row_bytes : 2 * share, &extra);
        const size_t smem = (sizeof(int) + sizeof(uint16_t) * kSortW) * p.bins[i];
        if (!launch_ahead(k_lookup_scatter, dim3(p.nch + extra), kSortBlock, smem, st, s, zs, i)) return TT_ERR_CUDA;
    }
    set_units(&a, VEC, kLkThreads);
    a.R = p.R;
    a.chunks = p.chunks;
    a.keys = p.keys[(p.passes - 1) & 1];
    a.pos = p.pos[(p.passes - 1) & 1];
    a.m = p.m;
    a.head = p.head;
    a.tail = p.tail;
    a.zero_first = cleared;
    const int64_t zero_blocks = (rows - cleared + a.zero_rows - 1) / a.zero_rows;
    const int per = kLkThreads / a.lanes;
    a.sum_blocks = (p.chunks + per - 1) / per * a.slices;
    if (!launch_ahead(k_lookup_sums<T, VEC>, dim3((unsigned)(a.sum_blocks + zero_blocks)), kLkThreads, 0, st, a)) return TT_ERR_CUDA;
    set_units(&a, VEC, 64);  // a popular id has dozens of partial sums: at least four threads to each column
    return launch_ahead(k_lookup_join<T, VEC>, dim3((unsigned)(p.chunks * a.slices)), kLkThreads, 0, st, a) ? TT_OK : TT_ERR_CUDA;
}

template <class T, int VEC>
tt_status run_lookup(const LookupArgs& a, const LookupPlan* plan, int sms, int dev, cudaStream_t st) {
    return plan ? backward_launch<T, VEC>(a, *plan, a.ids, sms, dev, st) : forward_launch<T, VEC>(a, st);
}

// The widest unit that divides the rows and on whose boundaries they begin.
template <class T>
tt_status run_lookup(const LookupArgs& a, const LookupPlan* plan, int sms, int dev, cudaStream_t st) {
    constexpr int e = (int)sizeof(T);
    auto fits = [&](int bytes) { return a.D * e % bytes == 0 && aligned(a.in, bytes) && aligned(a.out, bytes) && a.in_ld * e % bytes == 0 && a.out_ld * e % bytes == 0; };
    if (fits(16)) return run_lookup<T, 16 / e>(a, plan, sms, dev, st);
    if (fits(8)) return run_lookup<T, 8 / e>(a, plan, sms, dev, st);
    if (e == 2 && fits(4)) return run_lookup<T, e == 2 ? 2 : 1>(a, plan, sms, dev, st);
    return run_lookup<T, 1>(a, plan, sms, dev, st);
}

tt_status dispatch(int dtype, const LookupArgs& a, const LookupPlan* plan, int sms, int dev, cudaStream_t st) {
    if (dtype == TT_F32) return run_lookup<float>(a, plan, sms, dev, st);
    if (dtype == TT_BF16) return run_lookup<__nv_bfloat16>(a, plan, sms, dev, st);
    return run_lookup<__half>(a, plan, sms, dev, st);
}

}  // namespace
}  // namespace ttemb

using namespace ttemb;

extern "C" {

int64_t tt_emb_lookup_workspace(int64_t rows, int64_t vocab, int32_t dim, int32_t dtype) {
    if (lookup_sizes(rows, vocab, dim, dtype) != TT_OK) return -1;
    return (int64_t)lookup_plan(rows, vocab, dim, dtype, nullptr).bytes;
}

tt_status tt_emb_lookup_forward(const tt_lookup* lookup, void* out_dev, int64_t out_stride, int32_t* err_dev, tt_stream stream) {
    if (!lookup) return TT_ERR_ARG;
    const tt_lookup& l = *lookup;
    const tt_status s = lookup_sizes(l.rows, l.vocab, l.dim, l.dtype);
    if (s != TT_OK) return s;
    if (l.weight_stride < l.dim || out_stride < l.dim) return TT_ERR_SHAPE;
    if (!l.weight_dev || (l.rows && (!l.ids_dev || !out_dev))) return TT_ERR_ARG;
    if (!aligned(l.weight_dev, esize(l.dtype)) || !aligned(out_dev, esize(l.dtype)) || !aligned(l.ids_dev, 8) || !aligned(err_dev, 4)) return TT_ERR_ARG;
    if (l.rows == 0) return TT_OK;
    int dev = 0;
    const int sms = head_sms(&dev);
    if (sms <= 0) return TT_ERR_CUDA;
    LookupArgs a{};
    a.in = l.weight_dev;
    a.in_ld = l.weight_stride;
    a.out = out_dev;
    a.out_ld = out_stride;
    a.ids = l.ids_dev;
    a.N = l.rows;
    a.V = l.vocab;
    a.pad = -1;
    a.D = l.dim;
    a.scale = l.scale;
    a.err = err_dev;
    return dispatch(l.dtype, a, nullptr, sms, dev, reinterpret_cast<cudaStream_t>(stream));
}

tt_status tt_emb_lookup_backward(const tt_lookup* lookup, const void* grad_out_dev, int64_t grad_out_stride, void* grad_weight_dev,
                                 int64_t grad_weight_stride, int32_t accumulate, int32_t* err_dev, void* ws_dev, size_t ws_bytes,
                                 tt_stream stream) {
    if (!lookup) return TT_ERR_ARG;
    const tt_lookup& l = *lookup;
    const tt_status s = lookup_sizes(l.rows, l.vocab, l.dim, l.dtype);
    if (s != TT_OK) return s;
    if (grad_out_stride < l.dim || grad_weight_stride < l.dim) return TT_ERR_SHAPE;
    if (!grad_weight_dev || (l.rows && (!l.ids_dev || !grad_out_dev))) return TT_ERR_ARG;
    if (!aligned(grad_out_dev, esize(l.dtype)) || !aligned(grad_weight_dev, esize(l.dtype)) || !aligned(l.ids_dev, 8) || !aligned(err_dev, 4) ||
        !aligned(ws_dev, 256))
        return TT_ERR_ARG;
    const LookupPlan p = lookup_plan(l.rows, l.vocab, l.dim, l.dtype, ws_dev);
    if (ws_bytes < p.bytes || (p.bytes && !ws_dev)) return TT_ERR_ARG;
    int dev = 0;
    const int sms = head_sms(&dev);
    if (sms <= 0) return TT_ERR_CUDA;
    LookupArgs a{};
    a.in = grad_out_dev;
    a.in_ld = grad_out_stride;
    a.out = grad_weight_dev;
    a.out_ld = grad_weight_stride;
    a.ids = l.ids_dev;
    a.N = l.rows;
    a.V = l.vocab;
    a.pad = l.padding_idx;
    a.D = l.dim;
    a.scale = l.scale;
    a.accumulate = accumulate != 0;
    a.err = err_dev;
    return dispatch(l.dtype, a, &p, sms, dev, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
