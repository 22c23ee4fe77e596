/*
 * tt_emb.h -- C ABI of the GB300 (sm_103a) TT-EmbeddingBag library, libttemb.so.
 *
 * A TT-EmbeddingBag is a drop-in EmbeddingBag whose E x D table is held as
 * three tensor-train cores (TT-Rec / FBTT-Embedding pages; FBTT README,
 * opening paragraph and "How FBTT-Embedding works").  Row i, decoded as
 * i = i1 p2 p3 + i2 p3 + i3, is the chain product G1[i1] G2[i2] G3[i3]; the
 * rows named by each bag are sum- or mean-pooled (optionally weighted) into
 * one output row, and the backward pass applies a fused sparse SGD update to
 * the touched core slices (FBTT README, "Fused Kernel", sparse=True).
 *
 * Conventions for every entry point:
 *   - Pointers named *_dev are CUDA device pointers; the caller owns them and
 *     keeps them valid until the work queued on `stream` has completed.
 *   - Core k of a table is float32 [p_k][r_{k-1}][q_k][r_k] (r_0 = r_3 = 1),
 *     C-contiguous, so slice G_k[i_k] is contiguous.  The FBTT README's
 *     "Initialization" section gives the cores as r_{k-1} x p_k x q_k x r_k;
 *     the slice index is moved first here, which changes no value.
 *   - Column j of a row is j = j1 q2 q3 + j2 q3 + j3.
 *   - Bags are CSR: offsets_dev has num_bags + 1 int64 entries, offsets[0] = 0,
 *     offsets[num_bags] = nnz, non-decreasing; bag g holds the lookups
 *     offsets[g] .. offsets[g+1]-1.  (PyTorch's EmbeddingBag passes the B
 *     start positions only; append nnz to convert.)
 *   - A handle is not thread-safe; calls on one handle must be issued from
 *     one host thread and be ordered on the streams they are given.
 *   - No call throws; each returns a tt_status.  Host-side validation runs
 *     before anything is queued, and on failure nothing is modified.  Errors
 *     found on the device (an index outside [0, E), malformed offsets) are
 *     recorded in a sticky per-handle flag read by tt_emb_get_last_error();
 *     the offending lookups contribute nothing to the output, and a backward
 *     pass that follows such a forward pass leaves every core unchanged.
 */
#ifndef TT_EMB_H
#define TT_EMB_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct tt_emb tt_emb;          /* opaque handle */
typedef struct CUstream_st* tt_stream; /* same type as cudaStream_t; NULL = legacy default stream */

typedef enum {
    TT_OK = 0,
    TT_ERR_ARG = 1,     /* bad argument: null pointer, negative size, unknown mode */
    TT_ERR_SHAPE = 2,   /* inconsistent TT shape: p1 p2 p3 < E, q1 q2 q3 != D, rank <= 0, limits */
    TT_ERR_INDEX = 3,   /* device found an index outside [0, E) */
    TT_ERR_CUDA = 4,    /* a CUDA runtime call failed */
    TT_ERR_STATE = 5,   /* call out of order, e.g. backward without a forward */
    TT_ERR_TIMEOUT = 6, /* a bounded device wait gave up */
    TT_ERR_NOMEM = 7,   /* device workspace allocation failed */
    TT_ERR_BOUNDS = 8   /* debug build only (libttemb_debug.so): an internal index left its bound */
} tt_status;

typedef enum { TT_POOL_SUM = 0, TT_POOL_MEAN = 1 } tt_pool;

/* What tt_emb_backward does with the gradient g of each element of every
 * touched core slice (FBTT README, "Parameters": sparse, optimizer,
 * learning_rate, eps; "Fused Kernel"). */
typedef enum {
    TT_OPT_SGD = 0,     /* sparse=True, SGD:     G -= lr g                                   */
    TT_OPT_ADAGRAD = 1, /* sparse=True, Adagrad: s += g^2; G -= lr g / (sqrt(s) + eps)       */
    TT_OPT_GRAD = 2     /* sparse=False: the gradient is written out, the cores stay as they are */
} tt_optim;

/* Limits checked by the create calls. */
#define TT_MAX_P 1048576 /* each p_k */
#define TT_MAX_Q 64      /* each q_k */
#define TT_MAX_RANK 128  /* each r_k */
#define TT_MAX_D 256     /* q1 q2 q3 */

/* One table of a table-batched handle (FBTT README, "TableBatchedTTEmbeddingBag"). */
typedef struct {
    int64_t num_embeddings; /* E: rows of this table */
    int64_t p[3];           /* row factorisation, p1 p2 p3 >= E (FBTT README, "Parameters": tt_p_shapes) */
    int32_t q[3];           /* column factorisation, q1 q2 q3 = D (tt_q_shapes) */
    int32_t ranks[2];       /* r1, r2 (tt_ranks) */
    float* cores_dev[3];    /* caller-owned, 16-byte aligned device cores, updated in place by tt_emb_backward */
} tt_table_desc;

/*
 * Create a single-table handle.  FBTT README, "Parameters" (num_embeddings,
 * tt_p_shapes, tt_q_shapes, tt_ranks).  cores_dev[k] must hold
 * p_k * r_{k-1} * q_k * r_k floats and be 16-byte aligned (the kernels read
 * the cores as float4; a fresh cudaMalloc or torch allocation always is).
 * The handle keeps the core pointers (not
 * the data); the caller keeps the cores alive while the handle is used.
 * Device memory for the handle's fixed tables is allocated on the current
 * CUDA device, which every later call on the handle must also use.
 * Returns TT_ERR_ARG (null out/cores, misaligned cores), TT_ERR_SHAPE (see
 * limits above).
 */
tt_status tt_emb_create(int64_t num_embeddings, const int64_t p[3], const int32_t q[3],
                        const int32_t ranks[2], float* const cores_dev[3], tt_emb** out);

/*
 * Create a table-batched handle over num_tables >= 1 tables that share D
 * (FBTT README, "TableBatchedTTEmbeddingBag": many tables in one call; unlike
 * the README's version, the tables may differ in E, p, q and ranks).  Bags of
 * a batched call are ordered table-major: bag g = t * B + b is sample b of
 * table t, and its indices are row ids of table t.
 */
tt_status tt_emb_batch_create(int32_t num_tables, const tt_table_desc* descs, tt_emb** out);

/* Release the handle's device memory (not the caller's cores).  NULL is a no-op. */
void tt_emb_destroy(tt_emb* h);

/*
 * Size the handle's workspace for up to max_nnz lookups and max_bags bags, so
 * that later forward/backward calls within those sizes allocate nothing (and
 * may be captured in a CUDA graph).  Forward calls beyond the reserved sizes
 * grow the workspace themselves.
 */
tt_status tt_emb_reserve(tt_emb* h, int64_t max_nnz, int64_t max_bags);

/*
 * Forward pass (FBTT README, "How FBTT-Embedding works": forward(input,
 * offsets); the pooling of PyTorch's EmbeddingBag).
 *   indices_dev          int64 [nnz]          row ids (of the bag's table)
 *   offsets_dev          int64 [num_bags + 1] CSR bag boundaries
 *   per_sample_weights   float [nnz] or NULL   (NULL: every weight is 1)
 *   mode                 TT_POOL_SUM: out[g] = sum_n w_n row_n
 *                        TT_POOL_MEAN: out[g] = (1/L_g) sum_n w_n row_n, L_g = bag length
 *   out_dev              float [num_bags][D], written completely (empty bag: zeros)
 * num_bags must be a multiple of the handle's table count.  The decoded
 * lookups, their grouping and the partial products G1[i1] G2[i2] are kept in
 * the handle for the next tt_emb_backward().  Asynchronous on `stream`.
 * Returns TT_ERR_ARG (null pointers with nnz > 0, negative sizes, bad mode,
 * num_bags not a multiple of the table count), TT_ERR_NOMEM, TT_ERR_CUDA.
 */
tt_status tt_emb_forward(tt_emb* h, const int64_t* indices_dev, int64_t nnz,
                         const int64_t* offsets_dev, int64_t num_bags,
                         const float* per_sample_weights_dev, tt_pool mode, float* out_dev,
                         tt_stream stream);

/*
 * Backward pass fused with SGD (FBTT README, "Fused Kernel", sparse=True with
 * OptimType.SGD): for L = sum_g <out[g], grad_out[g]> of the most recent
 * forward pass on this handle, every touched slice becomes
 * G_k[s] - lr * dL/dG_k[s], all gradients taken at the pre-update cores;
 * no gradient is returned.  grad_out_dev is float [num_bags][D] of that
 * forward pass.  Consumes the saved forward state: a second backward without
 * a new forward returns TT_ERR_STATE.  If the forward pass recorded a device
 * error, no core is changed.  Asynchronous on `stream`.
 */
tt_status tt_emb_backward(tt_emb* h, const float* grad_out_dev, float lr, tt_stream stream);

/*
 * Choose the update that tt_emb_backward applies (default TT_OPT_SGD; the
 * tt_emb_backward description above is the SGD case).  FBTT README,
 * "Parameters": sparse selects between the fused update and returning the
 * core gradients to an external optimizer; optimizer and eps configure the
 * fused update.  No page fixes the Adagrad variant: this is element-wise
 * Adagrad with one accumulator per core element, lr_decay and weight decay 0.
 *   optim  TT_OPT_SGD, TT_OPT_ADAGRAD or TT_OPT_GRAD
 *   eps    Adagrad denominator term, finite and >= 0 (ignored otherwise)
 *   aux    3 * num_tables caller-owned device pointers, table-major
 *          (aux[3 t + k] belongs to core k of table t), each with the shape of
 *          that core, 16-byte aligned; NULL for TT_OPT_SGD.
 *            TT_OPT_ADAGRAD: the accumulators s, read and updated in place
 *              (a new run starts them at 0, or at an initial value >= 0);
 *            TT_OPT_GRAD: every tt_emb_backward overwrites the whole buffer
 *              with dL/dG_k (zeros for untouched slices).
 * The handle keeps the pointers, which must stay valid while it is used.
 * Synchronous (copies the handle's device tables); not for stream capture.
 * Returns TT_ERR_ARG (null handle, unknown optim, bad eps, null or misaligned
 * aux), TT_ERR_CUDA.
 */
tt_status tt_emb_set_optimizer(tt_emb* h, int32_t optim, float eps, float* const* aux);

/*
 * Update from summed gradients: the data-parallel step.  Bags are independent
 * in the forward pass and every core gradient is a sum over bags, so ranks that
 * hold disjoint shares of a batch's bags and identical cores can each run
 * tt_emb_forward + tt_emb_backward with TT_OPT_GRAD on their share, sum the
 * gradient buffers over the ranks (one all-reduce, outside this library), and
 * then apply the same update on every rank with this call; the cores then equal
 * those of one fused step over the whole batch, up to the order of summation.
 * The update rules are those of tt_emb_set_optimizer (FBTT README,
 * "Parameters": optimizer, learning_rate, eps; "Fused Kernel").
 *   optim      TT_OPT_SGD (G -= lr g) or TT_OPT_ADAGRAD (s += g^2;
 *              G -= lr g / (sqrt(s) + eps))
 *   grads_dev  3 * num_tables caller-owned device pointers (table-major, each
 *              shaped like its core, 16-byte aligned): the summed gradients
 *   state_dev  3 * num_tables Adagrad accumulators (same layout), updated in
 *              place; NULL for TT_OPT_SGD
 * An element whose summed gradient is exactly 0 keeps its bits (as every
 * element of an untouched slice does in the fused step).  An exact-copy
 * hot-row cache sees the changed slices as stale.  Allocates nothing;
 * asynchronous on `stream`.  Returns TT_ERR_ARG (null or misaligned
 * pointers, unknown optim, bad eps), TT_ERR_STATE (trainable cache rows,
 * whose gradients this call does not carry), TT_ERR_CUDA.
 */
tt_status tt_emb_apply_gradients(tt_emb* h, int32_t optim, float lr, float eps, float* const* grads_dev,
                                 float* const* state_dev, tt_stream stream);

/*
 * Expand rows [row0, row0 + nrows) of table `table` (0 for a single-table
 * handle) to a dense float [nrows][D] block (FBTT README,
 * "TableBatchedTTEmbeddingBag": expanding to full weight).  Row i of the table
 * is G1[i1] G2[i2] G3[i3] with i = i1 p2 p3 + i2 p3 + i3, read from the cores
 * as they are when the kernel runs.  out_dev is caller-owned, nrows * D
 * floats.  Asynchronous on `stream`.  Returns TT_ERR_ARG (null handle, null
 * out with nrows > 0, table out of range, rows outside [0, E)), TT_ERR_CUDA.
 */
tt_status tt_emb_full_weight(tt_emb* h, int32_t table, int64_t row0, int64_t nrows, float* out_dev,
                             tt_stream stream);

/*
 * Hot-row cache (FBTT README, "Software Cache"): decompress the n rows of
 * table 0 listed in rows_dev (n <= 2^29 int64 rows, distinct, within [0, E)) into a
 * device-resident fp32 cache, slot i holding the i-th smallest row (rows are
 * found through a hash index).  By default the cached rows are exact copies:
 * later forward passes read a cached row instead of contracting it, as long as
 * its three core slices have not changed since it was filled; a backward pass
 * marks the slices it updated and the next forward pass recomputes a stale row
 * (one lookup per row) and writes it back into the cache.  Results are the same
 * as without a cache.  With tt_emb_cache_set_trainable the rows are parameters
 * of their own, initialised here from the cores.  Replaces any previous cache
 * content; a forward pass made with the previous cache can no longer be
 * followed by a backward pass (TT_ERR_STATE) when its rows were trainable.
 * Synchronous.  Returns TT_ERR_ARG (bad n, rows, or a null pointer),
 * TT_ERR_STATE (a table-batched handle), TT_ERR_NOMEM, TT_ERR_CUDA.
 */
tt_status tt_emb_cache_populate(tt_emb* h, const int64_t* rows_dev, int64_t n, tt_stream stream);

/* Drop the cache and free its memory (also the LFU policy's cache; the access
 * counts stay).  Returns TT_ERR_ARG for a null handle. */
tt_status tt_emb_cache_disable(tt_emb* h);

/*
 * LFU cache policy (FBTT README, "Parameters": use_cache, cache_size,
 * hashtbl_size; "Software Cache": access frequencies are counted in an
 * open-addressing hash table during forward propagation, the cache is a
 * 32-way set-associative least-frequently-used cache, and it changes only
 * when it is populated, with values initialised from the TT cores).
 * Single-table handles only (TT_ERR_STATE otherwise).
 *
 * tt_emb_lfu_enable: allocate a frequency table of hashtbl_size entries (a
 *   power of two, 32 .. 2^30) and size the cache at cache_size rows rounded up
 *   to a multiple of 32 (cache_size / 32 sets of 32 ways).  From then on every
 *   forward pass counts each lookup's row: hash h = SplitMix64(row) (the first
 *   output of a SplitMix64 generator seeded with row), entry h mod hashtbl_size,
 *   linear probing over at most 64 entries; a row that finds no free or
 *   matching entry there is not counted.  Counting uses integer atomics, so
 *   the counts do not depend on the order of the lookups while the table has
 *   room.  Replaces any previous frequency table (counts start at 0).
 * tt_emb_lfu_populate: rebuild the cache from the counts: set k (k =
 *   (h >> 32) mod sets) holds the 32 most frequently counted rows whose hash
 *   maps to k (ties: the smaller row id); each cached value is computed from
 *   the cores.  By default cached rows are exact copies of TT rows: gradients
 *   go to the cores and a row whose slices change is recomputed on its next
 *   hit, so results equal the no-cache results.  With
 *   tt_emb_cache_set_trainable the cached rows are parameters of their own
 *   (see there).  Synchronous.
 * tt_emb_lfu_read: copy the counted (row, count) pairs, sorted by row, into
 *   caller-owned host arrays of cap entries; *n_out = number of pairs.
 * tt_emb_lfu_cached_rows: copy the cache's rows per slot (slot = set * 32 +
 *   way, -1 = empty way; or the sorted rows of tt_emb_cache_populate) into a
 *   host array of cap entries; *n_out = number of slots.  Synchronous.
 * tt_emb_lfu_disable: stop counting and free the frequency table.
 * Return TT_ERR_ARG (bad sizes, null pointers), TT_ERR_STATE (batched handle;
 * populate or read before enable), TT_ERR_NOMEM, TT_ERR_CUDA.
 */
tt_status tt_emb_lfu_enable(tt_emb* h, int64_t cache_size, int64_t hashtbl_size);
tt_status tt_emb_lfu_populate(tt_emb* h, tt_stream stream);
tt_status tt_emb_lfu_read(tt_emb* h, int64_t* rows_host, uint32_t* counts_host, int64_t cap, int64_t* n_out);
tt_status tt_emb_lfu_cached_rows(tt_emb* h, int64_t* rows_host, int64_t cap, int64_t* n_out);
tt_status tt_emb_lfu_disable(tt_emb* h);

/*
 * Trainable cache rows (FBTT README, "Parameters": sparse, where backward
 * gives the gradient w.r.t. the TT cores or the cache; "Software Cache":
 * cached rows are loaded without decompressing them).  Single-table handles
 * only (TT_ERR_STATE otherwise).
 *
 * tt_emb_cache_set_trainable(h, 1): from the next forward pass on, a lookup
 *   whose row is cached (a hit) reads the cached value instead of its TT row,
 *   and backward gives the hit's gradient to the cached value and none to the
 *   cores: the gradient of cached value [slot][j] is the sum over the hits of
 *   that slot of (the lookup's pooling scale: weight, divided by the bag
 *   length in mean mode) x grad_out[bag][j].  The sum is taken in 64-bit fixed
 *   point with integer atomics, so it does not depend on the order of the
 *   hits (each term, the fp32 product, is rounded to a step of 2^-S with
 *   |sum| < 2^62, S set by max|grad_out| x max|hit scale| and the lookup
 *   count).  The optimizer of
 *   tt_emb_set_optimizer then updates the cached values that some hit touched
 *   (SGD; Adagrad with its own state per cached value, zero at populate; or
 *   TT_OPT_GRAD, which keeps the gradient for tt_emb_cache_read and gives
 *   untouched values 0); misses train the cores as before.  Hits take no part
 *   in the TT contractions or their grouping: a core slice that only hits use
 *   is not touched.  The cache state (installed now or later by a populate
 *   call) is initialised from the cores.  (h, 0): back to exact-copy rows,
 *   recomputed from the cores now.  Synchronous.
 * tt_emb_cache_read: copy the cached values ([slots][D] fp32, slot order of
 *   tt_emb_lfu_cached_rows) into vals_dev and, trainable mode only, the last
 *   gradients of TT_OPT_GRAD into grads_dev (caller-owned device buffers; either
 *   may be NULL).  Stream-ordered.
 * tt_emb_cache_write: overwrite the cached values from vals_dev (same layout;
 *   trainable mode only: an external optimizer's step on the values after
 *   TT_OPT_GRAD).  Stream-ordered.
 * Return TT_ERR_ARG, TT_ERR_STATE (batched handle; grads_dev or a write
 * outside trainable mode), TT_ERR_NOMEM, TT_ERR_CUDA.
 */
tt_status tt_emb_cache_set_trainable(tt_emb* h, int32_t trainable, tt_stream stream);
tt_status tt_emb_cache_read(tt_emb* h, float* vals_dev, float* grads_dev, tt_stream stream);
tt_status tt_emb_cache_write(tt_emb* h, const float* vals_dev, tt_stream stream);

/*
 * Copy the decode of the most recent forward pass: for every lookup its
 * table, its slice indices (i1, i2, i3) and its bag.  Each *_dev is a
 * caller-owned int32 [nnz] device buffer; any may be NULL.  For checks.
 */
tt_status tt_emb_get_decoded(tt_emb* h, int32_t* table_dev, int32_t* i1_dev, int32_t* i2_dev,
                             int32_t* i3_dev, int32_t* bag_dev, tt_stream stream);

/*
 * Wait for the handle's queued work, then return and clear the sticky device
 * error (TT_ERR_INDEX, TT_ERR_ARG for malformed offsets, TT_ERR_TIMEOUT) or
 * TT_OK.  Returns TT_ERR_CUDA if the wait itself fails.
 */
tt_status tt_emb_get_last_error(tt_emb* h);

/*
 * Stage timing: when enabled, each forward/backward records a CUDA event
 * after each of its kernels on the call's stream.  tt_emb_stage_times()
 * waits for the last call and writes up to cap per-kernel durations in
 * milliseconds (kernel order of that call) with their names; returns the
 * number of kernels the call launched, or -1 on error.
 */
tt_status tt_emb_set_stage_timing(tt_emb* h, int enable);
int tt_emb_stage_times(tt_emb* h, int which /* 0 forward, 1 backward */, float* ms, const char** names,
                       int cap);

/* Kernels launched by the most recent forward (which = 0) or backward (1). */
int tt_emb_last_launch_count(tt_emb* h, int which);

/*
 * Bound of the handle's device waits.  The pages have no counterpart: the
 * tensor-core kernels wait for their own MMAs and for the bulk copies of their
 * G2 slices on mbarriers, at most `polls` polls (default 2^24, far longer than
 * any MMA batch or copy).  A wait that gives up records TT_ERR_TIMEOUT (read by
 * tt_emb_get_last_error), issues no further MMA, waits with the default bound
 * for the MMAs or copies already in flight and frees its tensor memory; the
 * call's results are then undefined and a following backward changes no core.  polls = 0 makes every such wait give up at once
 * (a test of that path).  Takes effect from the next call.  Returns
 * TT_ERR_ARG for a null handle.
 */
tt_status tt_emb_set_wait_limit(tt_emb* h, uint32_t polls);

/*
 * Forward pass that allocates no device memory.  The pages have no
 * counterpart: this entry point exists for callers that cannot call
 * cudaMalloc -- code running under a memory manager that owns all device
 * memory (a framework's caching allocator, a serving runtime with a fixed
 * budget), and code that must not synchronize the device or that runs while a
 * stream is captured into a CUDA graph.
 *
 * It computes what tt_emb_forward() computes for one table, without a handle:
 * the arguments mean what they mean for tt_emb_create() and tt_emb_forward()
 * (cores_dev are only read), and the caller owns every buffer.  err_dev, if
 * not NULL, is a caller-owned device int32 into which the kernel ORs 1 for an
 * index outside [0, E) (that lookup contributes nothing) and 2 for malformed
 * offsets; the caller clears it.  The only scratch is a static device array of
 * TT_NOALLOC_SCRATCH_BYTES that every GPU loading the library holds until the
 * process exits; one partial product of q1 q2 r2 floats per warp must fit in
 * it (TT_ERR_SHAPE otherwise).  Calls share that array, so calls whose work
 * overlaps on the GPU (unordered streams) race and give wrong results.  The
 * first call on a device looks up the array's device address (a CUDA runtime
 * call); make that first call before any stream capture.  Calls no cudaMalloc,
 * cudaFree or allocating library routine.  Asynchronous on `stream`.
 */
#define TT_NOALLOC_SCRATCH_BYTES (8 * 1024 * 1024)
tt_status tt_emb_forward_noalloc(int64_t num_embeddings, const int64_t p[3], const int32_t q[3],
                                 const int32_t ranks[2], const float* const cores_dev[3],
                                 const int64_t* indices_dev, int64_t nnz, const int64_t* offsets_dev,
                                 int64_t num_bags, const float* per_sample_weights_dev, tt_pool mode,
                                 float* out_dev, int32_t* err_dev, tt_stream stream);

/*
 * Vocabulary head: losses over the scores of rows against a whole table,
 *     z[n][v] = sum_d hidden[n][d] weight[v][d],
 * without an [N][V] array of them.  weight is any dense table: an output
 * projection, or the rows of a TT table (tt_emb_forward with one bag per row, whose
 * backward pass then takes the rows' gradient to the cores).  These calls need no
 * handle; every buffer is the caller's, and every call is asynchronous on `stream`
 * and allocates nothing (so it may be captured in a CUDA graph).
 */
typedef enum { TT_F32 = 0, TT_BF16 = 1, TT_F16 = 2 } tt_dtype;

/*
 * What the numbers keep.  Losses, lse, softmax statistics and sums are fp32.
 *   bf16, f16  enter the products as they are.  Scores for the losses are summed over 512
 *              columns in the tensor cores and beyond that with rounding; dz (below) is
 *              rounded to the type before the gradient products, whose sums run over a piece
 *              of the vocabulary (grad_hidden) or the rows (grad_weight) in the tensor cores,
 *              which cut low bits off: the gradients' error is some 1.4 times that of
 *              their own final rounding.
 *   fp32       an operand enters with 22 bits, or to 2^-39 of the largest finite magnitude
 *              under its scale where that is more: a hidden row (grad_weight: all that
 *              count), 128 x 128 elements of the table (dim <= 64: 256 rows), an x row of
 *              the 4-bit scores.  So one very large number (-1e9 in a column of biases) costs its
 *              neighbours bits; -inf does not.
 *   dz         fp32 and f16 are scaled by a power of two: grad_hidden keeps elements down to
 *              2^-28 (f16) or, with 22 bits, 2^-16 (fp32; 2^-39 absolute) of the row's own
 *              |grad_loss| T, rows down to 2^-100 of the heaviest; grad_weight loses what lies below
 *              2^-39 of the batch's largest |grad_loss| T.
 * Infinities are kept in every type: a table row that scores -inf drops out of lse and
 * grad_weight, as by a column of biases that hidden holds a 1 for; grad_hidden's column of
 * it is 0 times -inf, NaN, for rows that count.  An infinity times an infinity at one place is
 * NaN in fp32.  A score of +inf, and NaN, make lse NaN.
 */

#define TT_HEAD_MAX_ROWS 16777216    /* rows N */
#define TT_HEAD_MAX_VOCAB 1073741824 /* table rows V */
#define TT_HEAD_MAX_DIM 65536        /* width D */
#define TT_HEAD_MAX_TEACHER 1024     /* teacher entries per row; rows x entries < 2^31 */

typedef struct {
    const void* hidden_dev; /* [rows][dim], rows hidden_stride elements apart */
    const void* weight_dev; /* [vocab][dim], rows weight_stride elements apart */
    int64_t rows, vocab;
    int64_t hidden_stride, weight_stride; /* >= dim; elements of a row are contiguous */
    int32_t dim;
    int32_t dtype; /* tt_dtype of hidden and weight and of their gradients */
} tt_head;

/*
 * Bytes of workspace that a forward (backward = 0) or backward (1) call on `head`
 * needs; teacher_k: entries per row of the distillation calls, 1 for cross entropy.
 * The size depends on the shapes, the type, the device and on whether the rows are
 * 16-byte aligned (rows that are not, and fp32 rows, are copied).  The workspace is
 * 256-byte aligned and holds nothing between calls.  -1 for a head that the calls
 * would refuse.
 */
int64_t tt_emb_head_workspace(const tt_head* head, int32_t teacher_k, int32_t backward);

/*
 * Softmax cross entropy.
 *   targets_dev  int64 [rows]; a row whose target is ignore_index has loss 0 and
 *                gives no gradient (grad_hidden 0), whatever its hidden row and
 *                grad_loss hold
 *   loss_dev     float [rows]: lse[n] - z[n][targets[n]]
 *   lse_dev      float [rows]: log sum_v exp(z[n][v]), of every row
 *   err_dev      int32 or NULL; the call ORs in 1 for a target that is neither
 *                ignore_index nor in [0, vocab) (its row counts as ignored) and 4
 *                for a device wait that gave up (results undefined); the caller
 *                clears it
 * Backward: with lse from the forward call and grad_loss_dev float [rows] the
 * gradient of each row's loss,
 *   dz[n][v] = grad_loss[n] (exp(z[n][v] - lse[n]) - [v = targets[n]]),
 *   grad_hidden [rows][dim] = dz weight, grad_weight [vocab][dim] = dz^T hidden,
 * both written whole, contiguous, of the head's type.  The sums are taken in fp32
 * in an order that is fixed for given sizes: results repeat bit for bit.
 * Returns TT_ERR_ARG (null pointers, unknown type, misaligned or short workspace),
 * TT_ERR_SHAPE (limits above, stride < dim), TT_ERR_CUDA.
 */
tt_status tt_emb_xent_forward(const tt_head* head, const int64_t* targets_dev, int64_t ignore_index, float* loss_dev,
                              float* lse_dev, int32_t* err_dev, void* ws_dev, size_t ws_bytes, tt_stream stream);
tt_status tt_emb_xent_backward(const tt_head* head, const int64_t* targets_dev, int64_t ignore_index,
                               const float* lse_dev, const float* grad_loss_dev, void* grad_hidden_dev,
                               void* grad_weight_dev, int32_t* err_dev, void* ws_dev, size_t ws_bytes,
                               tt_stream stream);

/*
 * Distillation from a teacher's top logits.  Each row has teacher_k entries
 * (ids_dev int64 [rows][teacher_k], logits_dev float [rows][teacher_k]).  An entry
 * whose id is negative does not count, whatever its logit holds, nor does one whose
 * logit is -inf; an id >= vocab does not count and sets 1 in err_dev.  Over the
 * entries that count, q = softmax(logit / T); with lse[n] = log sum_v exp(z[n][v] / T)
 *   loss[n] = T^2 sum_k q[n][k] (log q[n][k] - z[n][id_k] / T + lse[n]),
 * the Kullback-Leibler divergence of the student from the teacher's renormalised
 * entries, scaled by T^2.  A row with no entry that counts has loss 0 and gives no
 * gradient.  Entries of a row with the same id add up in the gradient; in the loss
 * each keeps its own log q.  T in [1e-4, 1e4].  The teacher gets no gradient.
 * Backward: dz[n][v] = grad_loss[n] T (exp(z[n][v] / T - lse[n]) - sum of q of the
 * row's entries with id v), and the gradients as for cross entropy.  Errors as there.
 */
tt_status tt_emb_distill_forward(const tt_head* head, const int64_t* ids_dev, const float* logits_dev,
                                 int32_t teacher_k, float temperature, float* loss_dev, float* lse_dev,
                                 int32_t* err_dev, void* ws_dev, size_t ws_bytes, tt_stream stream);
tt_status tt_emb_distill_backward(const tt_head* head, const int64_t* ids_dev, const float* logits_dev,
                                  int32_t teacher_k, float temperature, const float* lse_dev,
                                  const float* grad_loss_dev, void* grad_hidden_dev, void* grad_weight_dev,
                                  int32_t* err_dev, void* ws_dev, size_t ws_bytes, tt_stream stream);

/*
 * Bound, in nanoseconds, of each wait inside the head's kernels (for their own
 * copies and MMAs; default 2e9).  Process-wide, from the next call on; 0 makes a wait
 * that is not already over give up, those of other threads' calls too (a test of that path).  A wait that gives up sets
 * 4 in err_dev; the call then ends with undefined results and leaves nothing running.
 */
tt_status tt_emb_head_set_wait_limit(uint64_t ns);

/*
 * Scores against a table held in 4 bits (serving):
 *   out[m][v] = sum_d scale[v][d / group] (code[v][d] - 8) x[m][d]
 * packed_dev: two codes to a byte, the even column in the low half, a row of
 * ceil(dim / 32) * 16 bytes (padding columns hold 8, which stands for 0), 16-byte
 * aligned.  scales_dev: bf16 bits [vocab][ceil(dim / group)].  group: 32, 64 or 128.
 *
 * tt_emb_q4_quantize lays a dense table out so: per group scale = bf16(max |w| / 7),
 *   code = round(w / scale) held within [-8, 7], plus 8; an all-zero group gets scale
 *   0.  A group with infinities gets an infinite scale and keeps only them (codes 7 and
 *   9), so they outweigh it; one with a NaN gets a scale of NaN.  weight_dev [vocab][dim] of `dtype` (tt_dtype), rows weight_stride apart.
 * tt_emb_q4_matvec: x_dev [rows][dim] of `dtype`, rows x_stride apart; out_dev float
 *   [rows][vocab], written whole.  Products with f16 and bf16 x are exact (bf16 values
 *   below 2^-31 of the row's largest lose bits), fp32 x enters with 22 bits; sums are
 *   fp32.  Meant for few rows: each 32 of them read the table once.
 * Both are asynchronous on `stream` and allocate nothing.  Return TT_ERR_ARG (null or
 * misaligned pointers, unknown type), TT_ERR_SHAPE (limits, group, stride), TT_ERR_CUDA.
 */
#define TT_Q4_MAX_ROWS 65536
tt_status tt_emb_q4_quantize(const void* weight_dev, int64_t weight_stride, int64_t vocab, int32_t dim,
                             int32_t dtype, int32_t group, uint8_t* packed_dev, uint16_t* scales_dev,
                             tt_stream stream);
tt_status tt_emb_q4_matvec(const void* x_dev, int64_t x_stride, int32_t rows, int32_t dtype,
                           const uint8_t* packed_dev, const uint16_t* scales_dev, int64_t vocab, int32_t dim,
                           int32_t group, float* out_dev, tt_stream stream);

/*
 * Rows of a dense table by id, times a scale, and the table's gradient:
 *     out[n][d] = scale weight[ids[n]][d]
 *     grad_weight[v][d] = scale sum of grad_out[n][d] over the n with ids[n] = v != padding_idx
 * The table is the kind that the vocabulary head scores (a tied table has both).  These
 * calls need no handle; every buffer is the caller's, every call is asynchronous on
 * `stream` and allocates nothing (so it may be captured in a CUDA graph).
 *   ids_dev      int64 [rows].  An id outside [0, vocab) gives a row of zeros, no gradient,
 *                and 1 in err_dev (int32 or NULL; the caller clears it)
 *   padding_idx  rows with this id give no gradient (forward: like any other); -1: none
 *   out          [rows][dim] of the table's type, rows out_stride elements apart; a product
 *                by the fp32 scale, rounded once
 *   grad_weight  [vocab][dim] of the table's type, rows grad_weight_stride apart.  accumulate
 *                0: every row written (rows that no id names with zeros).  1: added to the rows that
 *                are named, others neither read nor written: the gradient of a tied table, or,
 *                with the table itself and scale = -(learning rate) scale, its step of gradient
 *                descent.  Sums are fp32, rounded once, taken in an order that is fixed by
 *                the ids: results repeat bit for bit.
 * tt_emb_lookup_workspace: bytes of 256-byte aligned workspace that the backward call needs;
 * it holds nothing between calls.  -1 for sizes that the calls refuse.
 * Return TT_ERR_ARG (null or misaligned pointers, unknown type, short workspace),
 * TT_ERR_SHAPE (limits, stride < dim), TT_ERR_CUDA.
 */
#define TT_LOOKUP_MAX_ROWS 134217728 /* rows of a call; table rows and width as for the head */

typedef struct {
    const void* weight_dev; /* [vocab][dim], rows weight_stride elements apart; the backward call takes NULL */
    int64_t weight_stride;
    const int64_t* ids_dev;
    int64_t rows, vocab;
    int64_t padding_idx;
    int32_t dim;
    int32_t dtype; /* tt_dtype of weight, out and their gradients */
    float scale;
} tt_lookup;

int64_t tt_emb_lookup_workspace(int64_t rows, int64_t vocab, int32_t dim, int32_t dtype);
tt_status tt_emb_lookup_forward(const tt_lookup* lookup, void* out_dev, int64_t out_stride, int32_t* err_dev,
                                tt_stream stream);
tt_status tt_emb_lookup_backward(const tt_lookup* lookup, const void* grad_out_dev, int64_t grad_out_stride,
                                 void* grad_weight_dev, int64_t grad_weight_stride, int32_t accumulate,
                                 int32_t* err_dev, void* ws_dev, size_t ws_bytes, tt_stream stream);

/*
 * Losses of answers (sequences of sampled tokens) from the log probabilities of their tokens,
 * as the head gives them (minus its cross entropy), and the gradient of each of these.
 * Tokens lie one behind the other; sequence s holds offsets[s] .. offsets[s + 1] - 1, or, without
 * offsets, tokens / sequences tokens each (a padded batch).  A token whose mask is 0 does not
 * count, whatever its numbers are.  m[t] is 1 for a token that counts, n[s] how many do.
 * share[s] = 1 / n[s] if `average`, else 1 (a sequence without a token that counts: 0 for
 * every sum).  A token's terms are fp32 numbers; those of four neighbours (tokens 4 i .. 4 i + 3) are added in fp32, and
 * such groups in two floats (some 48 bits), whatever their number: of sums of differences at most
 * 3 x 2^-24 of the sum of their magnitudes is lost, and nothing of terms that are exact in groups of four.
 * Both need a workspace (256-byte aligned, nothing kept between calls) of tt_emb_answers_workspace bytes (-1: refused
 * sizes) forward; 0 bytes: none, NULL will do.
 *
 * Preference.  Sequences 0 .. P - 1 are chosen over sequences P .. 2 P - 1, pair by pair:
 *   rewards[s] = beta share[s] sum_t m[t] (logp[t] - reference[t])     (no reference: 0)
 *   margins[p] = h = rewards[p] - rewards[P + p] - margin
 *   loss[p] = -(1 - smoothing) log sigma(h) - smoothing log sigma(-h)  TT_PREF_SIGMOID
 *             max(0, 1 - h)                                            TT_PREF_HINGE
 *             ((h - 1/2) / beta)^2                                     TT_PREF_SQUARED
 *   (R. Rafailov et al., "Direct Preference Optimization", 2023; M. G. Azar et al., "A General
 *   Theoretical Paradigm to Understand Learning from Human Preferences", 2023.)
 *   Backward: grad_logp[t] = +-grad_loss[p] dloss/dh beta share[s] m[t]; reads margins and counts
 *   of the forward call, and of the tokens only the mask.
 *
 * Policy.  With d[t] = logp[t] - old[t], log_ratio[s] the mean of d over the tokens of s that count,
 * x[t] = log_ratio[s] (TT_POLICY_SEQUENCE) or d[t] (TT_POLICY_TOKEN), r = exp(x), advantage A
 * of the token or of its sequence:
 *   L[t] = -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A), and at most -dual_clip A where A < 0
 *          and dual_clip > 0
 *   k[t] with y = reference[t] - logp[t]:  -y (TT_KL_1), y^2 / 2 (TT_KL_2), exp(y) - 1 - y (TT_KL_3)
 *   kl[s] = share[s] sum_t m[t] k[t],  loss[s] = share[s] sum_t m[t] L[t] + kl_weight kl[s]
 *   clipped[s]: how many tokens that count have a ratio beyond the bound that holds for the
 *   sign of their A (none without a sign: 0, NaN).  Whether it is is decided on x itself (d is not rounded for that).
 *   No reference: k = 0.  TT_POLICY_SEQUENCE takes an advantage per sequence.
 *   (J. Schulman et al., "Proximal Policy Optimization Algorithms", 2017; D. Ye et al., "Mastering
 *   Complex Control in MOBA Games with Deep Reinforcement Learning", 2020: dual_clip; C. Zheng et al.,
 *   "Group Sequence Policy Optimization", 2025.)
 *   Backward: grad_logp[t] = grad_loss[s] share[s] m[t] (-A r [not clipped] + kl_weight dk/dlogp); reads
 *   log_ratio and counts of the forward call.  old, reference and advantages get no gradient.
 *
 * grad_logp is written whole (0 for tokens that do not count or lie behind the last
 * sequence).  err_dev (int32 or NULL; the caller clears it): 2 for offsets that do not begin
 * with 0, decrease, pass `tokens` or hold 2^31 tokens or more in one sequence (results undefined; no access outside the buffers).
 * Return TT_ERR_ARG (null or misaligned pointers, unknown kinds, numbers outside their ranges, short
 * workspace), TT_ERR_SHAPE (limits; no offsets and tokens no multiple of sequences), TT_ERR_CUDA.
 */
#define TT_ANSWERS_MAX_TOKENS 1099511627776 /* 2^40 */
#define TT_ANSWERS_MAX_SEQUENCES 16777216

typedef enum { TT_PREF_SIGMOID = 0, TT_PREF_HINGE = 1, TT_PREF_SQUARED = 2 } tt_pref_kind;
typedef enum { TT_POLICY_TOKEN = 0, TT_POLICY_SEQUENCE = 1 } tt_policy_level;
typedef enum { TT_KL_1 = 1, TT_KL_2 = 2, TT_KL_3 = 3 } tt_kl_kind;

typedef struct {
    const float* logp_dev;      /* [tokens]; the preference's backward call takes NULL */
    const float* reference_dev; /* [tokens] or NULL */
    const uint8_t* mask_dev;    /* [tokens], 0 or 1, or NULL: every token counts */
    const int64_t* offsets_dev; /* [sequences + 1] or NULL */
    int64_t tokens, sequences;
    int32_t average;
} tt_answers;

typedef struct {
    int32_t kind;           /* tt_pref_kind */
    double beta;            /* > 0 */
    double label_smoothing; /* in [0, 1); TT_PREF_SIGMOID only, else 0 */
    double margin;
} tt_preference;

typedef struct {
    const float* old_dev;        /* [tokens] */
    const float* advantages_dev; /* [tokens] if per_token, else [sequences] */
    int32_t per_token;
    int32_t level;     /* tt_policy_level */
    int32_t kl;        /* tt_kl_kind */
    double clip_low;   /* in [0, 1) */
    double clip_high;  /* >= 0 */
    double dual_clip;  /* 0 (none) or > 1 */
    double kl_weight;  /* >= 0 */
} tt_policy;

int64_t tt_emb_answers_workspace(int64_t tokens, int64_t sequences);
tt_status tt_emb_preference_forward(const tt_answers* answers, const tt_preference* how, float* loss_dev,
                                    float* margins_dev, float* rewards_dev, int32_t* counts_dev,
                                    int32_t* err_dev, void* ws_dev, size_t ws_bytes, tt_stream stream);
tt_status tt_emb_preference_backward(const tt_answers* answers, const tt_preference* how,
                                     const float* margins_dev, const int32_t* counts_dev,
                                     const float* grad_loss_dev, float* grad_logp_dev, tt_stream stream);
tt_status tt_emb_policy_forward(const tt_answers* answers, const tt_policy* how, float* loss_dev, float* kl_dev,
                                float* log_ratio_dev, int32_t* counts_dev, int32_t* clipped_dev,
                                int32_t* err_dev, void* ws_dev, size_t ws_bytes, tt_stream stream);
tt_status tt_emb_policy_backward(const tt_answers* answers, const tt_policy* how, const float* log_ratio_dev,
                                 const int32_t* counts_dev, const float* grad_loss_dev, float* grad_logp_dev,
                                 tt_stream stream);

/*
 * Scores against a table held in 8-bit integers (serving, evaluation):
 *   out[m][v] = xscale[m] scale[v] sum_d xcode[m][d] code[v][d]
 * with a scale for each row of x and each row of the table.  codes_dev: int8 [vocab][pitch], pitch =
 * ceil(dim / 16) * 16, 16-byte aligned; what padding columns hold does not matter.
 *
 * tt_emb_q8_quantize, of the rows of any matrix: scale = max |w| / 127 (fp32 division), code =
 *   127 w / max |w| rounded to nearest, ties to even, as if the quotient were exact; a row of
 *   zeros gets scale 0.  A row with infinities gets an infinite scale and keeps only them (codes 1
 *   and -1); one with a NaN gets a scale of NaN and codes 0.  Padding columns get 0.
 * tt_emb_q8_scores quantizes the rows of x in the same way, into its workspace, and multiplies.  The integer
 *   sums are exact; each is rounded once to fp32 and multiplied by the product of the two
 *   scales.  x_dev [rows][dim] of `dtype`, rows x_stride apart; out_dev float [rows][vocab], written whole.
 *   err_dev (int32 or NULL; the caller clears it): 4 for a device wait that gave up (results
 *   undefined; the bound is that of tt_emb_head_set_wait_limit).
 * tt_emb_q8_workspace: bytes of the 256-byte aligned workspace that the scores need; it holds nothing between
 * calls.  -1 for refused sizes.  All are asynchronous on `stream` and allocate nothing.  Return TT_ERR_ARG (null or
 * misaligned pointers, unknown type, short workspace), TT_ERR_SHAPE (limits, stride), TT_ERR_CUDA.
 */
#define TT_Q8_MAX_ROWS 16777216
int64_t tt_emb_q8_workspace(int64_t rows, int32_t dim);
tt_status tt_emb_q8_quantize(const void* weight_dev, int64_t weight_stride, int64_t rows, int32_t dim,
                             int32_t dtype, int8_t* codes_dev, float* scales_dev, tt_stream stream);
tt_status tt_emb_q8_scores(const void* x_dev, int64_t x_stride, int64_t rows, int32_t dtype,
                           const int8_t* codes_dev, const float* scales_dev, int64_t vocab, int32_t dim,
                           float* out_dev, int32_t* err_dev, void* ws_dev, size_t ws_bytes, tt_stream stream);

/* Static description of a status code; never NULL. */
const char* tt_emb_status_string(tt_status s);

#ifdef __cplusplus
}
#endif

#endif /* TT_EMB_H */
