/*
 * tp.h -- C ABI of the GB300 tensor-parallel sharded projection library (libtp.so).
 *
 * The method (diffusers documentation, "Tensor parallelism" page): every
 * weight matrix of a transformer block is split across tp_degree ranks,
 * either "colwise" (output features, weight dim 0: each rank computes a slice
 * of the output) or "rowwise" (input features, weight dim 1: each rank
 * computes a partial sum).  Fused projections are split block by block.  The
 * slices are joined at the layer boundary: concatenation (AllGather) for
 * colwise, summation (AllReduce) for rowwise.
 *
 * This library runs all tp_degree logical ranks on ONE GPU.  Every rank's
 * shard lives in its own buffer, every rank's GEMM runs inside one kernel
 * launch, and the joins happen in device memory inside the kernels.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Layout: every matrix is row-major and dense unless a leading dimension is
 *   given.  Weights use the nn.Linear layout [out_features, in_features];
 *   activations are [tokens, features].  Elements are bf16 (raw 16-bit
 *   patterns) unless stated; fp32 where stated.
 * - Ownership: the caller allocates and owns every buffer (inputs, outputs and
 *   workspace).  The library allocates no memory and keeps no pointer after a
 *   call returns.
 * - Asynchrony: kernels are enqueued on `stream` (a cudaStream_t; NULL is the
 *   legacy default stream) and the call returns without waiting.  Buffers
 *   must stay valid until the stream reaches that point.
 * - Validation: every argument is checked on the host before anything is
 *   copied or launched; a rejected call has no effect on device memory.  The
 *   plan checks follow the page's §Constraints and verification ("check both
 *   before loading or sharding any weight").
 * - Errors: a call returns a tp_status; TP_OK means the work was enqueued.
 *   tp_last_error() gives a message for the calling thread's last failure.
 *   Nothing falls back silently to another path (§Limitations: unsupported
 *   options raise instead of quietly doing something else).
 * - Device: the current CUDA device of the calling thread.  Requires sm_103a
 *   (GB300) for the GEMM entry points.
 */
#ifndef TP_H_
#define TP_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define TP_API __attribute__((visibility("default")))
#else
#define TP_API
#endif

typedef struct CUstream_st* tp_stream_t; /* same type as cudaStream_t */

typedef enum {
  TP_OK = 0,
  TP_ERR_INVALID_ARG = 1,         /* null pointer, negative size, rank outside [0, tp_degree), ... */
  TP_ERR_HEADS_NOT_DIVISIBLE = 2, /* tp_degree does not divide the attention-head count */
  TP_ERR_SPLIT_NOT_DIVISIBLE = 3, /* a packed block is not divisible by tp_degree on its own */
  TP_ERR_SPLIT_SUM = 4,           /* packed block sizes do not add up to the sharded dimension */
  TP_ERR_NOT_WHOLE_HEADS = 5,     /* a rank's part of a head-structured block is not whole heads */
  TP_ERR_ALIGNMENT = 6,           /* a pointer or row stride the kernels need 16-byte aligned is not */
  TP_ERR_NOT_PINNED = 7,          /* a host source pointer is pageable (not page-locked) memory */
  TP_ERR_WORKSPACE = 8,           /* workspace missing or smaller than tp_rowwise_workspace_bytes() */
  TP_ERR_CUDA = 9,                /* a CUDA runtime call failed (message in tp_last_error) */
  TP_ERR_TIMEOUT = 10,            /* a kernel gave up waiting on an internal barrier (tp_device_status) */
  TP_ERR_UNSUPPORTED = 11,        /* valid plan outside what this build implements (e.g. tp_degree > 16) */
  TP_ERR_IO = 12,                 /* a file could not be opened or read (tp_safetensors.h) */
  TP_ERR_FORMAT = 13,             /* a file is not a well-formed safetensors file (tp_safetensors.h) */
  TP_ERR_NOT_FOUND = 14           /* no tensor of that name in the file (tp_safetensors.h) */
} tp_status;

typedef enum { TP_COLWISE = 0, TP_ROWWISE = 1 } tp_style;
typedef enum { TP_GATHER = 0, TP_REDUCE = 1 } tp_combine_mode;
typedef enum { TP_ACT_NONE = 0, TP_ACT_GELU_TANH = 1, TP_ACT_SWIGLU = 2 } tp_act;
/* Flag OR'd into tp_linear_colwise's act argument: chunked fp32 accumulation (see there). */
#define TP_ACCUM_CHUNKED 0x100
typedef enum {
  TP_REDUCE_NONE = 0,      /* write every rank's fp32 partial; join later with tp_combine(TP_REDUCE) */
  TP_REDUCE_WORKSPACE = 1, /* fp32 partials to a workspace, summed in the GEMM epilogue by the ranks */
  TP_REDUCE_ACCUM = 2      /* each tile's ranks accumulate in turn into one fp32 on-chip accumulator */
} tp_reduce_mode;

#define TP_MAX_DEGREE 16 /* largest tp_degree the GEMM entry points accept */
#define TP_MAX_SPLITS 16 /* largest number of packed blocks in one weight */

/* ------------------------------------------------------------------------ */
/* Plan                                                                      */
/* ------------------------------------------------------------------------ */

/*
 * tp_validate -- check a sharding plan for one weight [rows, cols].
 *
 * "Tensor parallelism" page: §Load a sharded model (tp_degree must divide the
 * number of attention heads), §Fused projections (packed blocks, absolute
 * sizes as stored in _tp_packed_col_blocks / _tp_packed_row_blocks) and
 * §Constraints and verification (every packed block divisible by tp_degree
 * on its own).  Checks, in order:
 *   1. TP_ERR_INVALID_ARG: tp_degree >= 1, rows/cols/num_heads/head_dim >= 0,
 *      style valid, 0 <= n_splits <= TP_MAX_SPLITS, fused_splits non-NULL when
 *      n_splits > 0, every split > 0.
 *   2. TP_ERR_HEADS_NOT_DIVISIBLE: num_heads > 0 and num_heads % tp_degree != 0.
 *   3. TP_ERR_SPLIT_SUM: the splits do not add up to the sharded dimension
 *      (rows for TP_COLWISE, cols for TP_ROWWISE).
 *   4. TP_ERR_SPLIT_NOT_DIVISIBLE: some split % tp_degree != 0.
 *   5. TP_ERR_NOT_WHOLE_HEADS: head_dim > 0 and some (split / tp_degree) %
 *      head_dim != 0 (the sharded dimension is made of heads of head_dim).
 * fused_splits: host array of n_splits absolute block sizes along the sharded
 * dimension, in packed order; NULL/0 means one block (a plain split).
 * Pure host function; touches no device.
 */
TP_API tp_status tp_validate(int64_t rows, int64_t cols, tp_style style, int tp_degree, int64_t num_heads,
                      int64_t head_dim, const int64_t* fused_splits, int n_splits);

/*
 * tp_shard_shape -- shape of every rank's dense shard after tp_validate's
 * checks 1, 3 and 4: [rows / tp_degree, cols] for TP_COLWISE, [rows, cols /
 * tp_degree] for TP_ROWWISE.  out_rows/out_cols: host pointers, written on
 * TP_OK only.  Pure host function.
 */
TP_API tp_status tp_shard_shape(int64_t rows, int64_t cols, tp_style style, int tp_degree,
                         const int64_t* fused_splits, int n_splits, int64_t* out_rows, int64_t* out_cols);

/* ------------------------------------------------------------------------ */
/* Shard extraction                                                          */
/* ------------------------------------------------------------------------ */

/*
 * tp_plan_shard -- copy rank `rank`'s slice of a bf16 weight into a dense
 * device buffer.
 *
 * "Tensor parallelism" page, §Load a sharded model: each rank reads only its
 * own slice of every weight and places it directly on its device, so no
 * full-size weight is ever staged there; §Limitations: enable_parallelism()
 * shards a model already in memory.  Both are this call: `weight` may be
 * page-locked host memory (the slice is read over the CPU-GPU link straight
 * into `dev_out` by the copy engines, one transfer per packed block -- a
 * column window of every row for TP_ROWWISE -- so no SM is taken from kernels
 * running beside the load; nothing else reaches the device) or device memory
 * (a device-to-device copy kernel).  Pageable host memory is rejected with
 * TP_ERR_NOT_PINNED.
 *
 * Slice definition (§Colwise and rowwise, §Fused projections): with packed
 * blocks of sizes s_0..s_{n-1} at offsets o_b along the sharded dimension,
 * block b contributes [o_b + rank*s_b/p, o_b + (rank+1)*s_b/p) and the parts
 * are concatenated in block order.  TP_COLWISE slices rows, TP_ROWWISE slices
 * columns.  A fused QKV weight with splits {H,H,H} thus gives rank r the rows
 * [Q_r; K_r; V_r] of whole heads; a gate/up weight with {F,F} gives
 * [gate_r; up_r].
 *
 * weight:  bf16 [rows, cols] row-major (host page-locked or device).
 * dev_out: device buffer of tp_shard_shape() elements, dense row-major.
 * num_heads/head_dim: as in tp_validate (0 to skip those checks).
 * The copy is bit-exact (any 16-bit pattern, NaN payloads included).
 * Errors: everything tp_validate returns, TP_ERR_INVALID_ARG for NULL
 * pointers with a non-empty shard or a dev_out that is not device memory,
 * TP_ERR_NOT_PINNED, TP_ERR_CUDA.
 */
TP_API tp_status tp_plan_shard(const void* weight, int64_t rows, int64_t cols, tp_style style, int tp_degree, int rank,
                        const int64_t* fused_splits, int n_splits, int64_t num_heads, int64_t head_dim,
                        void* dev_out, tp_stream_t stream);

/*
 * tp_plan_shard_ranks -- tp_plan_shard for ranks [rank_begin, rank_begin +
 * rank_count) in one launch: dev_outs is a host array of rank_count device
 * buffers, dev_outs[i] receiving rank (rank_begin + i)'s shard.  Same slice
 * definition, checks, sources and errors as tp_plan_shard; the range must lie
 * in [0, tp_degree).  rank_count == 0 validates the plan and copies nothing.
 * This is how one process that plays every rank loads all their shards.
 */
TP_API tp_status tp_plan_shard_ranks(const void* weight, int64_t rows, int64_t cols, tp_style style, int tp_degree,
                                     int rank_begin, int rank_count, const int64_t* fused_splits, int n_splits,
                                     int64_t num_heads, int64_t head_dim, void* const* dev_outs, tp_stream_t stream);

/*
 * tp_plan_shard_many -- several extractions (e.g. every weight of a block) in
 * as few launches as possible: every request is a tp_plan_shard_ranks call,
 * with the same slice definition, checks and errors.  All requests are
 * checked before anything is copied; a refused request leaves every output
 * untouched and the error message names the request's index.  Requests from
 * device memory share one copy-kernel launch (more only beyond 64 copy
 * segments: one per packed block per rank); requests from page-locked host
 * memory are one copy-engine transfer per segment.  1 <= n_requests <= TP_MAX_SHARD_REQUESTS (0 is a no-op);
 * `requests` and the arrays it points to are read during the call only.
 */
#define TP_MAX_SHARD_REQUESTS 64
typedef struct {
  const void* weight;           /* bf16 [rows, cols] row-major: page-locked host or device memory */
  int64_t rows, cols;
  tp_style style;
  int tp_degree;
  int rank_begin, rank_count;   /* ranks [rank_begin, rank_begin + rank_count) */
  const int64_t* fused_splits;  /* NULL, or n_splits absolute packed block sizes */
  int n_splits;
  int64_t num_heads, head_dim;  /* as in tp_validate (0 skips the check) */
  void* const* dev_outs;        /* host array of rank_count device buffers */
} tp_shard_request;
TP_API tp_status tp_plan_shard_many(const tp_shard_request* requests, int n_requests, tp_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Sharded projections                                                       */
/* ------------------------------------------------------------------------ */

/*
 * tp_linear_colwise -- every rank's colwise projection in one launch:
 *     Y_r = act(X . W_r^T + b_r)      for r = 0 .. tp_degree-1
 *
 * "Tensor parallelism" page, §Colwise and rowwise: the input X is replicated
 * and each rank computes its slice of the output features; the output stays
 * sharded for the rowwise projection that follows.
 *
 * x:           device bf16 [T, K] (shared by every rank).
 * w_shards:    host array of tp_degree device pointers, each bf16 [N_r, K]
 *              (the dense shards tp_plan_shard writes).
 * bias_shards: NULL, or host array of tp_degree device pointers (each NULL or
 *              bf16 [N_r], sharded like the weight's rows).
 * act:         TP_ACT_NONE / TP_ACT_GELU_TANH (0.5x(1+tanh(sqrt(2/pi)(x+0.044715x^3))))
 *              / TP_ACT_SWIGLU (the shard is [gate_r; up_r], N_r even, and
 *              Y_r = silu(gate) * up has N_r/2 columns).  The activation is
 *              applied to the fp32 accumulator before rounding to bf16.
 * y_shards:    host array of tp_degree device pointers, each bf16 [T, N_out]
 *              with row stride ldy elements (N_out = N_r, or N_r/2 for SwiGLU).
 *              ldy = 0 means N_out (dense).  Passing y_shards[r] = Y + r*N_out
 *              with ldy = tp_degree*N_out writes the gathered (AllGather)
 *              output [T, tp_degree*N_out] directly.
 * Accumulation is fp32; outputs are rounded to nearest-even bf16.
 * act | TP_ACCUM_CHUNKED (TP_ACT_NONE only; TP_ERR_UNSUPPORTED otherwise):
 *              the tensor core adds each step of 16 products into its fp32
 *              accumulator without rounding to nearest, so a long K sum drifts:
 *              over K = 6144 about 0.35 % of the bf16 outputs round to the
 *              other neighbour of the exact value (0.02 % for a sum rounded to
 *              nearest at every step).  With this flag the products are summed
 *              on the tensor core in chunks of K = 1024, each from zero, and
 *              the chunks are added in fp32 with round-to-nearest by the
 *              epilogue, which brings it to about 0.07 %.  Use it where the
 *              output feeds a step that amplifies one-ulp differences -- the
 *              Q, K and V of attention, whose softmax turns a rounding flip in
 *              a key into a change of every query's weights.  It costs about
 *              9 % of the projection's time (8 epilogue warps keep the running
 *              sums in registers; the accumulator is handed to them once per
 *              chunk instead of once per tile).
 * Alignment (TP_ERR_ALIGNMENT): K % 8 == 0, N_out % 8 == 0, ldy % 8 == 0 and
 * every pointer 16-byte aligned.  tp_degree <= TP_MAX_DEGREE.
 * T == 0 or N_r == 0 enqueues nothing and returns TP_OK.
 */
TP_API tp_status tp_linear_colwise(const void* x, const void* const* w_shards, const void* const* bias_shards, tp_act act,
                            int tp_degree, int64_t T, int64_t K, int64_t N_r, void* const* y_shards, int64_t ldy,
                            tp_stream_t stream);

/*
 * tp_linear_rowwise -- every rank's rowwise projection and the sum of the
 * partials in one launch:
 *     P_r = X_r . W_r^T ,  Z = sum_r P_r (+ bias, once)
 *
 * "Tensor parallelism" page, §Colwise and rowwise: each rank computes a
 * partial sum from its slice of the input features, and one AllReduce at the
 * block boundary (after the colwise -> rowwise pair) rebuilds the result.
 * The partials are summed in rank order, in fp32.
 *
 * x_shards: host array of tp_degree device pointers, each bf16 [T, K_r]
 *           (rank r's slice of the input features, e.g. the colwise output).
 * w_shards: host array of tp_degree device pointers, each bf16 [N, K_r].
 * bias:     NULL or device bf16 [N]; added once, after the sum.
 * mode:
 *   TP_REDUCE_ACCUM: for each output tile, rank 0's, then rank 1's, ...
 *     products accumulate into one fp32 tensor-memory accumulator; out is
 *     bf16 [T, N].  No workspace (ws_bytes may be 0).
 *   TP_REDUCE_WORKSPACE: each rank's fp32 partial tile goes to `workspace`
 *     and is counted on a per-tile atomic counter; when all tp_degree partials
 *     of a tile are in (a bounded wait; the launch is cooperative so the ranks'
 *     CTAs are resident together), each rank sums its 1/tp_degree share of the
 *     tile's rows in rank order and writes bf16 [T, N] to out.  Needs
 *     ws_bytes >= tp_rowwise_workspace_bytes(...).  The counters are cleared on
 *     `stream` by the call itself.
 *   TP_REDUCE_NONE: out is fp32 [tp_degree][T][N], rank r's partial (the bias,
 *     if any, is added to rank 0's partial only); join with tp_combine.
 * Alignment (TP_ERR_ALIGNMENT): K_r % 8 == 0, N % 8 == 0, pointers 16-byte
 * aligned.  tp_degree <= TP_MAX_DEGREE.  T == 0 or N == 0 enqueues nothing.
 * Calls that share a workspace must not overlap on the GPU.
 */
TP_API tp_status tp_linear_rowwise(const void* const* x_shards, const void* const* w_shards, const void* bias, int tp_degree,
                            int64_t T, int64_t K_r, int64_t N, tp_reduce_mode mode, void* workspace, size_t ws_bytes,
                            void* out, tp_stream_t stream);

/*
 * tp_linear_rowwise_split_input -- the "rowwise_split_input" style: a rowwise
 * projection whose input is replicated on every rank, each rank computing its
 * partial from its own slice of that input.
 *
 * "Tensor parallelism" page, §Colwise and rowwise table: "rowwise_split_input"
 * shards the input features (weight dim 1) and each rank computes a partial
 * result from its slice of the replicated input and its weights; the sum
 * gives every rank all output features (for a standalone projection reading a
 * replicated activation, e.g. an AdaLN modulation projection).
 *     Z = sum_r X[:, r*K/p : (r+1)*K/p] . W_r^T (+ bias, once)
 *
 * x: device bf16 [T, K] with row stride ldx elements (0 = K); rank r reads
 *    columns [r*K/p, (r+1)*K/p) in place (no copy).
 * w_shards: host array of tp_degree device pointers, each bf16 [N, K/p] (the
 *    plain rowwise shards).  bias, mode, workspace, out: as tp_linear_rowwise.
 * Errors: TP_ERR_SPLIT_NOT_DIVISIBLE if tp_degree does not divide K; the
 * alignment rules of tp_linear_rowwise with K/p and ldx multiples of 8.
 */
TP_API tp_status tp_linear_rowwise_split_input(const void* x, int64_t ldx, const void* const* w_shards,
                                               const void* bias, int tp_degree, int64_t T, int64_t K, int64_t N,
                                               tp_reduce_mode mode, void* workspace, size_t ws_bytes, void* out,
                                               tp_stream_t stream);

/* Bytes of device workspace tp_linear_rowwise needs for `mode` (0 unless TP_REDUCE_WORKSPACE). */
TP_API size_t tp_rowwise_workspace_bytes(int tp_degree, int64_t T, int64_t N, tp_reduce_mode mode);

/* Size of the library's built-in scratch array used by tp_linear_rowwise_noalloc (64 MiB per GPU). */
#define TP_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/*
 * tp_linear_rowwise_noalloc -- tp_linear_rowwise in TP_REDUCE_WORKSPACE mode,
 * for callers that cannot allocate device memory.  The pages have no
 * counterpart of this call; it exists for the host program, not the method.
 *
 * Who needs it: code that runs where allocating is not allowed or not
 * possible -- for instance a plug-in called by a framework that owns all
 * device memory and hands out none, or a process whose memory was claimed up
 * front by a pool so that a new cudaMalloc would fail (cudaMalloc can also
 * stall the whole device, which latency-bound callers must avoid).  Such a
 * caller still passes its inputs and output; the fp32 partials and tile
 * counters live in one fixed array compiled into this library
 * (TP_NOALLOC_SCRATCH_BYTES of device memory, held by every GPU that loads the
 * library until the process exits).
 *
 * Arguments, layout, result and numerics are those of tp_linear_rowwise with
 * mode TP_REDUCE_WORKSPACE: x_shards/w_shards are host arrays of tp_degree
 * device pointers (bf16 [T, K_r] and [N, K_r]), bias is NULL or bf16 [N]
 * (added once), out is bf16 [T, N].
 * Limits: the call is refused with TP_ERR_WORKSPACE, before any device work,
 * when tp_rowwise_workspace_bytes(tp_degree, T, N, TP_REDUCE_WORKSPACE)
 * exceeds TP_NOALLOC_SCRATCH_BYTES (roughly tp_degree * T * N <= 16M).
 * When the memory is claimed: the array belongs to the library's GEMM
 * module, and the CUDA driver claims its device memory when it loads that
 * module on a device -- with lazy module loading (the default) at the first
 * call on that device that launches one of the library's GEMMs or looks the
 * array up (this call).  A caller whose memory pool will claim the device's
 * free memory should make one call of this entry point on each device (any
 * small problem, e.g. T = 1) before the pool does; from then on no call
 * claims memory.
 * The first call on a device (and the first in a new CUDA context, e.g.
 * after cudaDeviceReset) looks up the array's device address with that
 * device current; make that first call before any stream capture.  No
 * allocation happens in this call or the ones it makes.
 * Every call uses the same array and it keeps the last call's contents; the
 * call clears the tile counters itself.  Calls whose kernels overlap on the
 * GPU (other streams, other threads) race on the array: serialise them.
 */
TP_API tp_status tp_linear_rowwise_noalloc(const void* const* x_shards, const void* const* w_shards, const void* bias,
                                           int tp_degree, int64_t T, int64_t K_r, int64_t N, void* out,
                                           tp_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Attention over a rank's local heads                                       */
/* ------------------------------------------------------------------------ */

/*
 * tp_attention_heads -- attention of one rank over its local heads:
 *     O_h = softmax(Q_h K_h^T / sqrt(head_dim)) V_h     for h < n_heads
 *
 * "Tensor parallelism" page, §Colwise and rowwise: the colwise Q, K and V
 * projections give each rank a subset of heads (tp_degree divides the head
 * count), so the rank attends over them alone and its output feeds its
 * rowwise out-projection directly.  No mask, no positional embedding; head h
 * occupies columns [h*head_dim, (h+1)*head_dim) of each of Q, K and V.
 *
 * qkv:  device bf16 [T, 3*n_heads*head_dim] with row stride ld_qkv elements
 *       (0 = dense): Q, then K, then V -- the rank's colwise QKV output.
 * out:  device bf16 [T, n_heads*head_dim] with row stride ldo (0 = dense).
 * workspace: device buffer of tp_attention_workspace_bytes(T, n_heads,
 *       head_dim) bytes, owned by the caller; none (NULL, 0) at head_dim 64 and
 *       128, where the fused kernel reads Q, K and V in place; for other head
 *       sizes V^T (each group of 8 keys twice) and the fp32 scores of up to
 *       16 heads at a time.
 * Scores and softmax are fp32; the probabilities enter the P.V product (fp32
 * accumulation) as two bf16 terms, P_hi (P truncated to bf16 in the fused
 * kernel of head_dim 64 and 128, rounded elsewhere) and P_lo = bf16(P - P_hi), which
 * carry P to about 2^-16 relative (one bf16 term would carry 2^-9, an error
 * that the block's later bf16 roundings amplify); O is rounded to bf16.
 * Alignment (TP_ERR_ALIGNMENT): T, head_dim, ld_qkv, ldo multiples of 8, pointers
 * 16-byte aligned.  T == 0 enqueues nothing.  TP_ERR_WORKSPACE if too small.
 */
TP_API tp_status tp_attention_heads(const void* qkv, int64_t ld_qkv, int64_t T, int n_heads, int head_dim,
                                    void* workspace, size_t ws_bytes, void* out, int64_t ldo, tp_stream_t stream);

/* Bytes of device workspace tp_attention_heads needs (0 at head_dim 64 and 128). */
TP_API size_t tp_attention_workspace_bytes(int64_t T, int n_heads, int head_dim);

/*
 * tp_attention_heads_ranks -- tp_attention_heads for n_ranks ranks in one
 * call: qkv[r] and out[r] (host arrays of n_ranks device pointers) are rank
 * r's QKV output and attention output, every rank with the same T, n_heads,
 * head_dim, ld_qkv and ldo.  With head_dim 64 or 128 one kernel launch covers every
 * rank's heads, so a small per-rank head count still fills the GPU, and no
 * workspace is needed; other head sizes run the ranks one after another
 * through the same workspace.  Same arithmetic, checks and errors as
 * tp_attention_heads; 1 <= n_ranks <= TP_MAX_DEGREE (TP_ERR_UNSUPPORTED above).
 * workspace: tp_attention_ranks_workspace_bytes(n_ranks, T, n_heads, head_dim).
 */
TP_API tp_status tp_attention_heads_ranks(int n_ranks, const void* const* qkv, int64_t ld_qkv, int64_t T, int n_heads,
                                          int head_dim, void* workspace, size_t ws_bytes, void* const* out,
                                          int64_t ldo, tp_stream_t stream);

/* Bytes of device workspace tp_attention_heads_ranks needs (0 at head_dim 64 and 128, and for an empty or
 * invalid call). */
TP_API size_t tp_attention_ranks_workspace_bytes(int n_ranks, int64_t T, int n_heads, int head_dim);

/* ------------------------------------------------------------------------ */
/* Join                                                                      */
/* ------------------------------------------------------------------------ */

/*
 * tp_combine -- join per-rank results in device memory (the page's opening
 * paragraph: "an AllReduce or AllGather at the layer boundary").
 *   TP_GATHER: partials[r] is bf16 [T, N_each]; out is bf16 [T, tp_degree*N_each]
 *              with columns [r*N_each, (r+1)*N_each) taken from rank r.  Bit-exact.
 *   TP_REDUCE: partials[r] is fp32 [T, N_each]; out is bf16 [T, N_each] =
 *              round_nearest_even(sum_r partials[r]), summed in rank order in fp32.
 * partials: host array of tp_degree device pointers.  out: device buffer.
 * Any alignment is accepted (16-byte aligned rows take the vector path).
 */
TP_API tp_status tp_combine(tp_combine_mode mode, const void* const* partials, int tp_degree, int64_t T, int64_t N_each,
                     void* out, tp_stream_t stream);

/* ------------------------------------------------------------------------ */
/* 8-bit projections                                                         */
/* ------------------------------------------------------------------------ */

/*
 * The block-scaled 8-bit format of the calls below: e4m3 codes (1 byte) with
 * one power-of-two scale per group of 128, held as an e8m0 byte (scale =
 * 2^(byte - 127), 255 = NaN).  An activation's groups are 128 consecutive
 * features of one token: scales [T, ceil(K/128)].  A weight's groups are its
 * 128 x 128 blocks: scales [ceil(rows/128), ceil(K/128)].  The last group of a
 * row or column may be shorter.  The pages have no counterpart of these calls:
 * they load and run the model in bf16; here the same shards, projections and
 * joins run with half the weight bytes and twice the tensor-core rate.
 *
 * A weight is quantised shard by shard (after tp_plan_shard), so that a
 * shard's blocks start at its own first row and column.
 */

/*
 * tp_quantize_fp8 -- codes and scales of a bf16 matrix:
 *     e = ceil(log2(max|x| / 448)) over a group, clamped to [-127, 127]
 *         (0 for a group of zeros),  scale byte = e + 127,
 *     q = e4m3(x / 2^e), rounded once, to nearest even.
 * A group that holds a NaN or an infinity becomes NaN: byte 255 and NaN codes.
 *
 * x:      device bf16 [rows, cols], row stride ldx elements (0 = cols).
 * block_rows: 1 (groups of 128 features of one row: activations) or 128
 *         (128 x 128 blocks: weights).
 * q:      device e4m3 [rows, cols], row stride ldq (0 = cols).
 * scales: device e8m0 [ceil(rows/block_rows), ceil(cols/128)], row stride lds
 *         (0 = dense).  Any alignment; 4-byte aligned rows are read faster by
 *         the projections.
 * Alignment (TP_ERR_ALIGNMENT): cols % 16 == 0, ldx % 8 == 0, ldq % 16 == 0,
 * x and q 16-byte aligned.  q and scales must overlap neither x nor each other.
 * rows == 0 or cols == 0 enqueues nothing and returns TP_OK.
 */
TP_API tp_status tp_quantize_fp8(const void* x, int64_t ldx, int64_t rows, int64_t cols, int block_rows, void* q,
                                 int64_t ldq, void* scales, int64_t lds, tp_stream_t stream);

/*
 * tp_linear_colwise_fp8 -- tp_linear_colwise on the 8-bit format, every rank
 * in one launch:  Y_r = act(X . W_r^T + b_r), X and W_r the values their codes
 * and scales stand for.
 *
 * x, x_scales: device e4m3 [T, K] with row stride ldx (0 = K) and e8m0
 *              [T, ceil(K/128)] with row stride ld_xs (0 = dense), shared by
 *              every rank.
 * w_shards, w_scales: host arrays of tp_degree device pointers, each e4m3
 *              [N_r, K] and e8m0 [ceil(N_r/128), ceil(K/128)], dense.
 * bias_shards: NULL, or host array of tp_degree device pointers (each NULL or
 *              bf16 [N_r]).
 * act:         as tp_linear_colwise (SwiGLU shards are [gate_r; up_r]; N_r/2
 *              need not be a multiple of 128), applied to the fp32 sum.
 * y_shards:    host array of tp_degree device pointers, row stride ldy
 *              elements (0 = N_out).  With y_scales NULL each is bf16
 *              [T, N_out] (and the gathered layout of tp_linear_colwise works).
 * y_scales:    NULL, or host array of tp_degree device pointers: Y_r then
 *              leaves as e4m3 [T, N_out] with e8m0 [T, ceil(N_out/128)] (row
 *              stride ld_ys, 0 = dense), quantised from the unrounded fp32
 *              values as tp_quantize_fp8 does with block_rows 1 -- the input
 *              tp_linear_rowwise_fp8 takes.
 * The sum over K is one fp32 accumulator of the tensor core, scales applied
 * inside; with few tokens K may be split over up to 8 accumulators that are
 * added in fp32 in K order.  The same call gives the same bits every time.
 * Alignment (TP_ERR_ALIGNMENT): K and ldx % 16 == 0; N_out and ldy % 8 == 0
 * (% 16 with y_scales); x, w_shards, y_shards 16-byte aligned, bias_shards 2-byte.
 * T == 0 or N_r == 0 enqueues nothing and returns TP_OK.  No output may overlap an input
 * or another output.
 */
TP_API tp_status tp_linear_colwise_fp8(const void* x, int64_t ldx, const void* x_scales, int64_t ld_xs,
                                       const void* const* w_shards, const void* const* w_scales,
                                       const void* const* bias_shards, tp_act act, int tp_degree, int64_t T, int64_t K,
                                       int64_t N_r, void* const* y_shards, int64_t ldy, void* const* y_scales,
                                       int64_t ld_ys, tp_stream_t stream);

/*
 * tp_linear_rowwise_fp8 -- tp_linear_rowwise (its on-chip sum) on the 8-bit
 * format:  Z = sum_r X_r . W_r^T (+ bias, once), in rank order, in fp32.
 *
 * x_shards, x_scales: host arrays of tp_degree device pointers, each e4m3
 *         [T, K_r] with row stride ldx (0 = K_r) and e8m0 [T, ceil(K_r/128)]
 *         with row stride ld_xs (0 = dense) -- what tp_linear_colwise_fp8
 *         writes with y_scales.  A replicated input [T, p*K_r] is passed as p
 *         pointers into it (with K_r % 128 == 0, so that no group is shared).
 * w_shards, w_scales: host arrays of tp_degree device pointers, each e4m3
 *         [N, K_r] and e8m0 [ceil(N/128), ceil(K_r/128)], dense.
 * bias:   NULL or device bf16 [N]; added once, after the sum.
 * out:    device bf16 [T, N], row stride ldo elements (0 = N).
 * Alignment (TP_ERR_ALIGNMENT): K_r and ldx % 16 == 0, N and ldo % 8 == 0,
 * x_shards, w_shards and out 16-byte aligned, bias 2-byte.  Accumulation as tp_linear_colwise_fp8.
 * T == 0 or N == 0 enqueues nothing and returns TP_OK.  No output may overlap an input
 * or another output.
 */
TP_API tp_status tp_linear_rowwise_fp8(const void* const* x_shards, int64_t ldx, const void* const* x_scales,
                                       int64_t ld_xs, const void* const* w_shards, const void* const* w_scales,
                                       const void* bias, int tp_degree, int64_t T, int64_t K_r, int64_t N, void* out,
                                       int64_t ldo, tp_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Between sharded blocks                                                    */
/* ------------------------------------------------------------------------ */

typedef enum { TP_NORM_NONE = 0, TP_NORM_RMS = 1, TP_NORM_LAYER = 2 } tp_norm;

#define TP_NORM_MAX_D 32768 /* widest row tp_residual_norm accepts */

/*
 * tp_residual_norm -- what stands between one sharded block and the next,
 * each row read once:
 *     h = alpha * x + gate * post_norm(y)          (the residual stream)
 *     u = norm(h) * (1 + scale) + shift            (the next block's input)
 * Norms and modulations are replicated modules of the model, outside the
 * sharding plan ("Tensor parallelism" page, §What to leave out): every rank
 * computes the same rows, so one call serves them all.
 *
 *     rms(v)   = v / sqrt(mean(v^2) + eps) * weight + bias
 *     layer(v) = (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps) * weight + bias
 * (weight and bias optional), over the D elements of a row.  Everything is
 * fp32 until an output is stored; u is computed from the unrounded h.  Squares
 * and their sums are fp32 too: a row whose squares add up past 3.4e38 norms to
 * zeros (NaN where it holds an infinity).
 *
 * Without a branch (y NULL; h, gate and post_norm unset) u = norm(alpha * x) *
 * (1 + scale) + shift.  Without u (u NULL; norm, scale, shift and u_scales
 * unset) only h is written.  h may be x itself with the same row stride (the
 * residual updated in place); no other overlap of an output with an input or
 * another output.
 *
 * gate, scale and shift (each optional) are [mod_rows, D] tables with the row
 * stride ld_mod: row t of the call uses table row t / rows_per_mod.
 * mod_rows = 1 with rows_per_mod = T is one vector for every row;
 * rows_per_mod = 1 is a row per token.
 * u_scales set: u is e4m3 with e8m0 scales [T, ceil(D/128)], quantised from
 * the unrounded fp32 values as tp_quantize_fp8 does with block_rows 1.
 * Row strides of 0 mean dense rows.
 * Errors: TP_ERR_INVALID_ARG for sizes, strides and combinations outside the
 * above (and mod_rows * rows_per_mod < T); TP_ERR_ALIGNMENT unless D and every
 * row stride but ld_u_scales are multiples of 8 (D and ldu of 16 with u_scales)
 * and every pointer but u_scales is 16-byte aligned; TP_ERR_UNSUPPORTED above
 * TP_NORM_MAX_D.  T == 0 or D == 0 enqueues nothing and returns TP_OK.
 */
typedef struct {
  int64_t T, D;
  const void* x;            /* bf16 [T, D] */
  int64_t ldx;
  const void* y;            /* NULL, or bf16 [T, D]: the block's output */
  int64_t ldy;
  tp_norm post_norm;
  const void *post_weight, *post_bias; /* NULL, or bf16 [D] */
  float alpha;
  float eps;                /* of both norms */
  const void *gate, *scale, *shift;    /* NULL, or bf16 [mod_rows, D] */
  int64_t ld_mod, mod_rows, rows_per_mod;
  void* h;                  /* NULL, or bf16 [T, D] */
  int64_t ldh;
  tp_norm norm;
  const void *weight, *bias;           /* NULL, or bf16 [D] */
  void* u;                  /* NULL, or bf16 [T, D] (e4m3 with u_scales) */
  int64_t ldu;
  void* u_scales;           /* NULL, or e8m0 [T, ceil(D/128)] */
  int64_t ld_u_scales;
} tp_residual_norm_args;
TP_API tp_status tp_residual_norm(const tp_residual_norm_args* args, tp_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Paged 8-bit cache of keys and values                                      */
/* ------------------------------------------------------------------------ */

/*
 * Serving a sharded transformer: each rank keeps the keys and values of its
 * own KV heads ("Tensor parallelism" page, §Colwise and rowwise: the colwise
 * Q, K and V projections give each rank a subset of heads) in pages of
 * page_size tokens, in the 8-bit format above with one scale for each page and
 * head.  The pages have no counterpart of these calls (they describe no cache).
 *
 * One decoding step or prompt chunk of a rank is
 *     tp_linear_colwise(_fp8) -> Q, K, V columns   (bf16)
 *     tp_kv_append_fp8        -> Q rotated, K rotated and cached, V cached
 *     tp_attention_paged_fp8  -> attention over the cache
 *     tp_linear_rowwise       -> the out-projection.
 *
 * Cache.  k[r] and v[r] are rank r's codes, e4m3 [n_pages, n_kv_heads,
 * page_size, head_dim] with ld_page elements from page to page (0 = dense);
 * k_scales[r] and v_scales[r] are e8m0 [n_pages, n_kv_heads] with ld_scales
 * from page to page (0 = n_kv_heads).  head_dim is 64 or 128, page_size 16, 32,
 * 64 or 128 (TP_ERR_UNSUPPORTED otherwise).  Codes are 16-byte aligned and
 * ld_page is a multiple of 16 (TP_ERR_ALIGNMENT); scales have any alignment.
 * No initial value is needed: a page is only read where tokens were appended.
 *
 * Batch.  Every rank serves the same sequences.  seq_start (n_seqs + 1 entries,
 * ascending from seq_start[0] >= 0 to at most T), kv_len (n_seqs) and
 * page_table (n_seqs rows of max_pages, row stride ld_table, 0 = max_pages)
 * are int32 in DEVICE memory, read when the kernels run, so that a captured
 * CUDA graph takes the values of each replay.  Sequence s has the new rows
 * [seq_start[s], seq_start[s+1]), at most max_new of them, and kv_len[s] tokens
 * with the new ones; its row i of n stands at position kv_len[s] - n + i, and
 * position j is slot j % page_size of page page_table[s][j / page_size].  Rows
 * of T outside every sequence (padding) are neither read nor written.  A page
 * may be in several sequences' tables (a shared prefix), but not be appended
 * to by two in one call.  Table entries of pages that no row of the call sees
 * (behind kv_len, or before every row's window) may hold anything.
 *
 * What only the device can see is checked there: a token without a place (a
 * negative position, a page outside the table or the cache) is not cached, a
 * key in such a page is not seen, a token whose rotation is outside its table
 * is NaN, rows beyond max_new are left out, and so is the whole of a sequence
 * whose rows do not ascend within [0, T] or whose length is below 0 or above 2^30.
 * Nothing is read or written out of bounds, and tp_device_status reports
 * TP_ERR_INVALID_ARG.
 *
 * Sizes (TP_ERR_UNSUPPORTED beyond): 2^30 rows, pages, and keys of a sequence,
 * 65535 heads of a rank, 2^24 sequences; for the attention also 65535 KV heads
 * of all ranks, and page tables of 2^40 keys over all of them.
 */
typedef struct {
  int n_ranks;                  /* 1 .. TP_MAX_DEGREE */
  int n_kv_heads;               /* of one rank */
  int head_dim, page_size;
  int64_t n_pages;
  void* const* k;               /* host arrays of n_ranks device pointers */
  void* const* v;
  void* const* k_scales;
  void* const* v_scales;
  int64_t ld_page, ld_scales;
} tp_paged_cache;

typedef struct {
  int n_seqs;
  int max_new;                  /* at least the new rows of any sequence */
  const int32_t* seq_start;     /* device [n_seqs + 1] */
  const int32_t* kv_len;        /* device [n_seqs] */
  const int32_t* page_table;    /* device [n_seqs, max_pages] */
  int64_t ld_table, max_pages;
} tp_paged_batch;

/* Which elements of a head form a pair: x[i] and x[i + rot_dim/2], or x[2i] and x[2i + 1]. */
typedef enum { TP_ROPE_HALF = 0, TP_ROPE_PAIRS = 1 } tp_rope_style;

/*
 * The position rotation of Q and K: pair i of a token becomes
 * (x1 c_i - x2 s_i, x2 c_i + x1 s_i) with the row [c_0 .. c_{rot_dim/2 - 1},
 * s_0 ..] of cos_sin that belongs to the token: row `position`, or row
 * positions[t] of its row t.  Elements from rot_dim on stay as they are.  The
 * table is the caller's (any base, scaling or number of axes; computed in
 * double precision, far positions keep their angles).
 */
typedef struct {
  tp_rope_style style;
  int rot_dim;                  /* multiple of 16, at most head_dim */
  const float* cos_sin;         /* device [n_positions, rot_dim], 16-byte aligned */
  int64_t ld;                   /* row stride in elements, multiple of 4; 0 = rot_dim */
  int64_t n_positions;
  const int32_t* positions;     /* NULL, or device [T] */
} tp_rope;

/*
 * tp_kv_append_fp8 -- every rank's new tokens into its cache, and their Q
 * rotated, in one launch.
 *
 * qkv[r]: device bf16 [T, (n_heads + 2 n_kv_heads) head_dim], row stride
 *         ld_qkv (0 = dense): rank r's Q, K and V columns.
 * rope:   NULL (no rotation), or the rotation of Q and K.
 * q_out:  NULL (Q is left alone), or host array of device pointers, each bf16
 *         [T, n_heads head_dim] with row stride ld_q (0 = dense): Q rotated in
 *         fp32 and rounded once.  q_out[r] may be qkv[r] with ld_q = ld_qkv (Q rotated
 *         in place); no other output may overlap an input or another output.
 *
 * K (rotated in fp32, not rounded in between) and V are quantised by page and
 * head: e is the least exponent >= -127 with max|x| <= 448 * 2^e over the new
 * tokens of the page, and not less than the page's own where older tokens of
 * the sequence are in it; the scale byte is e + 127 and a new code is
 * e4m3(x / 2^e), rounded once to nearest even.  Where e grew, the older
 * tokens' codes q become e4m3(q * 2^(e_old - e)) (exact but for codes that
 * become subnormal).  A page with a NaN or an infinity becomes NaN for that
 * head (byte 255, NaN codes).  Slots behind the last token are left as they
 * were.  Appending the same tokens again changes nothing, and a token's
 * cache does not depend on what else is in the batch.
 * Alignment (TP_ERR_ALIGNMENT): ld_qkv and ld_q % 8 == 0, qkv and q_out 16-byte.
 * T == 0, n_seqs == 0 or max_new == 0 enqueues nothing.
 */
TP_API tp_status tp_kv_append_fp8(const tp_paged_cache* cache, const tp_paged_batch* batch, const void* const* qkv,
                                  int64_t ld_qkv, int64_t T, int n_heads, const tp_rope* rope, void* const* q_out,
                                  int64_t ld_q, tp_stream_t stream);

/*
 * tp_attention_paged_fp8 -- attention of every rank's new tokens over its cache:
 *     O_h = softmax(scale * Q_h K_g^T) V_g,  g = h / (n_heads / n_kv_heads)
 * K and V the values their codes and scales stand for.  A token at position p
 * sees the keys j < kv_len of its sequence with j <= p (causal) and
 * j > p - window (window > 0, causal only); a row that sees no key is 0.
 *
 * q:    host array of device pointers, each bf16 [T, n_heads head_dim] with row
 *       stride ld_q (0 = dense); n_heads is a multiple of n_kv_heads.
 * out:  host array of device pointers, each bf16 [T, n_heads head_dim] with row
 *       stride ldo (0 = dense); may not overlap q or another output.
 * workspace: device buffer of tp_attention_paged_workspace_bytes(...) bytes,
 *       16-byte aligned, owned by the caller, of any content.  Calls that share one must not
 *       overlap on the GPU.
 * Codes and Q enter the tensor cores as fp16, scaled by powers of two.  Of a row of Q, what lies 2^-39 below its
 * largest element is lost.  With up to 32 rows a KV head (see below) K enters exactly, and a key's
 * probability times value is off by at most 2^-30 of the largest V scale met so far.  With more rows K enters relative to
 * the largest K scale among 128 keys and V to the largest V scale so far, those of keys that a row does not see
 * among them: an element is off by at most 2^-32 of that scale, a page whose scale is 2^32 or more below it enters as
 * 0, and a probability is off by 2^-31 of the row's largest.  Products, softmax and sums are fp32 (in the tensor core
 * without rounding to nearest, in pieces of at most 2^19 keys), the probabilities
 * enter P.V as fp16 (besides the above 2^-11 relative, an eighth of the output's own 2^-8).  A
 * page whose K or V is NaN (scale byte 255, as tp_kv_append_fp8 leaves it) makes the rows that see
 * it NaN and no others; NaN codes in a page with another scale byte may make any row of
 * the sequence NaN.  The same call gives the same bits every time.
 * One kernel serves a call, chosen by max_new * n_heads / n_kv_heads: up to 32 rows a KV head, or more.  The one for
 * more takes two to three times as long for single tokens, so a step with a chunk of a prompt beside many decoding
 * sequences is best two calls (64 sequences 117 us and a chunk of 300 45, together 309).
 * Alignment (TP_ERR_ALIGNMENT): ld_q and ldo % 8 == 0, q and out 16-byte.
 * T == 0, n_seqs == 0 or max_new == 0 enqueues nothing.
 */
TP_API tp_status tp_attention_paged_fp8(const tp_paged_cache* cache, const tp_paged_batch* batch, const void* const* q,
                                        int64_t ld_q, int64_t T, int n_heads, float scale, int causal, int window,
                                        void* workspace, size_t ws_bytes, void* const* out, int64_t ldo,
                                        tp_stream_t stream);

/* Bytes of device workspace tp_attention_paged_fp8 needs on the current device (0 for a call that it would
 * refuse or that enqueues nothing). */
TP_API size_t tp_attention_paged_workspace_bytes(const tp_paged_cache* cache, const tp_paged_batch* batch, int64_t T,
                                                 int n_heads);

/* ------------------------------------------------------------------------ */
/* Diagnostics                                                               */
/* ------------------------------------------------------------------------ */

/* Message for the calling thread's last failed call ("" if none).  Valid until the thread's next call. */
TP_API const char* tp_last_error(void);

/* Name of a status code ("TP_OK", "TP_ERR_ALIGNMENT", ...). */
TP_API const char* tp_status_name(tp_status status);

/*
 * tp_device_status -- synchronise `stream`, then report whether any kernel of
 * this library on the current device gave up on an internal wait (every wait
 * is bounded; a kernel that gives up records it and exits cleanly) or met an
 * index in device memory that it could not use (the paged cache's calls).
 * Returns TP_ERR_TIMEOUT or TP_ERR_INVALID_ARG and clears the record if so, TP_ERR_CUDA if the stream
 * reported an error, TP_OK otherwise.
 */
TP_API tp_status tp_device_status(tp_stream_t stream);

/*
 * tp_set_tile_wait_limit_ns -- how long a CTA of a TP_REDUCE_WORKSPACE call
 * waits for the other ranks' partials of its output tile (the one wait of the
 * library on other CTAs) before it gives up: it then records TP_ERR_TIMEOUT
 * for tp_device_status, skips its share of the tile's sums, drains its copies
 * and MMAs and exits.  The output of such a call is not valid.  0 restores
 * the default of 2 s.  The value is read when a call enqueues its kernel, so
 * it applies to calls made after this one (and a captured CUDA graph keeps the
 * value of its capture).  Process-wide; the waits of a CTA on its own copies
 * and MMAs keep a fixed bound of 2 s.  Exists so that the give-up path can be
 * exercised: a budget far below the time the ranks of a tile take to arrive
 * makes the wait run out without any fault.
 */
TP_API void tp_set_tile_wait_limit_ns(uint64_t ns);

/* The current tile-wait bound in nanoseconds (see tp_set_tile_wait_limit_ns). */
TP_API uint64_t tp_tile_wait_limit_ns(void);

/* Library ABI version (major * 100 + minor). */
TP_API int tp_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* TP_H_ */
