/*
 * mse.h -- C ABI of the GB300 (sm_103a) shared-expert SwiGLU MLP library.
 *
 * The library computes, on one GPU:
 *   - the Kimi-K3 shared-expert / dense SwiGLU MLP
 *       y = W_down . ( SiLU(W_gate . x) * (W_up . x) )
 *     with a merged gate_up weight (gate rows first), hidden 7168 and
 *     intermediate 6144 in bf16
 *     ("[Kimi-K3] Add option to shard the shared expert instead of replicating",
 *      sections "Problem" and "Change");
 *   - the tensor-parallel sharded form of that MLP: shard r of tp owns the
 *     intermediate slice [r*s, (r+1)*s), s = I/tp, computes a partial output over
 *     it for all gathered tokens, and the partials are summed -- the sum half of
 *     the reduce-scatter; rank r keeps token rows [r*T/tp, (r+1)*T/tp)
 *     (same page, section "Change"; prhub analysis of vllm PR #50656, sections
 *      "实现拆解" and "关键源码片段");
 *   - the merged MLA q_a/kv_a latent projection stored as tensor-parallel
 *     column shards, whose gathered output is rank-major and is restored to the
 *     logical [q_a | kv_a] layout
 *     ("[II] TP-shard Kimi MLA latent projections", sections "Behavior",
 *      "Technical reason" and "Compatibility").
 *
 * Conventions (every entry point):
 *   - bf16 tensors are uint16_t bit patterns; all tensors are dense row-major.
 *   - Every tensor pointer is a DEVICE pointer owned by the caller.  The library
 *     allocates no device memory; scratch comes from the caller's workspace.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *     Launches are asynchronous on it; nothing synchronises.
 *   - The return value reports host-side validation and launch errors.  Errors
 *     raised on the device (a bounded wait that ran out) are reported later by
 *     mse_poll_device_error().
 *   - Arguments are validated before any CUDA call, so invalid calls fail the
 *     same way with or without a GPU.  There is no CPU fallback: on a device
 *     other than sm_103 the calls return MSE_ERR_UNSUPPORTED_DEVICE.
 *   - "capacity" arguments are element counts of the caller's buffer; a buffer
 *     smaller than the geometry needs is rejected as MSE_ERR_GEOMETRY (the
 *     truncated-geometry rejection of the MLA page, section "Validation").
 *   - The library is thread-safe; calls on the same stream are ordered.
 */
#ifndef MSE_H
#define MSE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Exported symbols (the library is built with hidden default visibility). */
#if defined(__GNUC__)
#define MSE_API __attribute__((visibility("default")))
#else
#define MSE_API
#endif

typedef uint16_t mse_bf16;

typedef enum {
    MSE_OK = 0,
    MSE_ERR_INVALID_ARG = 1,        /* null pointer, non-positive size, bad enum      */
    MSE_ERR_NOT_DIVISIBLE = 2,      /* I, H, q or kv not divisible by tp; T by parts  */
    MSE_ERR_GEOMETRY = 3,           /* capacity too small, rank range outside [0,tp)  */
    MSE_ERR_WORKSPACE = 4,          /* workspace missing, too small or misaligned     */
    MSE_ERR_UNSUPPORTED_DEVICE = 5, /* no CUDA device, or not compute capability 10.3 */
    MSE_ERR_CUDA = 6,               /* a CUDA runtime call failed                      */
    MSE_ERR_TIMEOUT = 7,            /* a device-side bounded wait ran out              */
    MSE_ERR_UNSUPPORTED_SHAPE = 8   /* kernel path forced by mse_set_kernel_path()
                                       cannot serve this shape/alignment               */
} mse_status;

typedef enum { MSE_BF16 = 0, MSE_F32 = 1 } mse_dtype;

/* Kernel path selection (process-wide; default MSE_PATH_AUTO).
 *   AUTO:        tensor-core (tcgen05/TMA) kernels where the shape and the
 *                16-byte alignment allow, else the generic CUDA-core kernels.
 *   GENERIC:     always the generic CUDA-core kernels (any shape).
 *   TENSORCORE:  always tcgen05 kernels; calls they cannot serve return
 *                MSE_ERR_UNSUPPORTED_SHAPE. */
typedef enum { MSE_PATH_AUTO = 0, MSE_PATH_GENERIC = 1, MSE_PATH_TENSORCORE = 2 } mse_kernel_path;

/* Tensor-core kernel for the token counts the decode-size kernels do not serve
 * (MSE_TUNE_SWAPAB_MAX_T), process-wide.
 *   AUTO:   CTA-pair kernel (two SMs share one 256 x 256 tile) up to 256 tokens and from
 *           512 on, single-CTA 128 x 256 kernel between.
 *   SINGLE: always the single-CTA kernel.   PAIR: always the CTA-pair kernel. */
typedef enum { MSE_PREFILL_AUTO = 0, MSE_PREFILL_SINGLE = 1, MSE_PREFILL_PAIR = 2 } mse_prefill_kernel;

/* ---------------------------------------------------------------------------
 * Workspace sizing.  The workspace holds the bf16 intermediate h [T x I] and,
 * for the tensor-core path, fp32 split-K partial tiles and the sync words (tile
 * counters and flags).  It must be 256-byte aligned and ZERO-FILLED before its
 * first use.  The sync words sit at the END of the buffer (their size depends on
 * H and I, or on q_dim + kv_dim, only); h and the partial tiles are laid out from
 * its start.  Every call that completes leaves the sync words zero again, so a
 * workspace of mlp_swiglu_workspace_bytes(T, H, I) bytes serves any sequence of
 * calls on one stream with at most T tokens and the same H and I (likewise for
 * the merged projection).  A call with another H or I needs a freshly zeroed
 * workspace.  Calls that run concurrently (different streams) need different
 * workspaces.  After MSE_ERR_TIMEOUT the caller must zero the workspace again.
 * A call accepts any workspace at least as large as its own minimal need, which
 * can be smaller than the size query's answer (the query covers all smaller T).
 * ------------------------------------------------------------------------- */

/* Bytes of a workspace that serves mlp_swiglu_forward, mlp_swiglu_shard_partial
 * and mlp_swiglu_shard_forward for every token count up to T (tp does not change
 * it).  Returns 0 on invalid arguments. */
MSE_API size_t mlp_swiglu_workspace_bytes(int64_t T, int64_t H, int64_t I);

/* Bytes of a workspace that serves merged_proj_forward for every token count up
 * to T with the same q_dim + kv_dim.  Returns 0 on invalid arguments. */
MSE_API size_t merged_proj_workspace_bytes(int64_t T, int64_t H, int64_t q_dim, int64_t kv_dim);

/* Byte range [*offset, *offset + *bytes) of the sync words (tile counters and
 * flags) inside a workspace of workspace_bytes for calls with at most T tokens
 * and this H and I.  Only this range must be zero before a call: after
 * MSE_ERR_TIMEOUT, zeroing it is enough to reuse the workspace.  Returns
 * MSE_ERR_WORKSPACE when workspace_bytes is below the call's minimal need,
 * MSE_ERR_INVALID_ARG on invalid sizes or null pointers.  Host only. */
MSE_API mse_status mlp_swiglu_workspace_sync_range(int64_t T, int64_t H, int64_t I, size_t workspace_bytes,
                                                   size_t *offset, size_t *bytes);

/* The same for a merged-projection workspace (the tile counters). */
MSE_API mse_status merged_proj_workspace_sync_range(int64_t T, int64_t H, int64_t q_dim, int64_t kv_dim,
                                                    size_t workspace_bytes, size_t *offset, size_t *bytes);

/* ---------------------------------------------------------------------------
 * Replicated SwiGLU MLP ("[Kimi-K3] Add option to shard the shared expert
 * instead of replicating", section "Change": gate_up projection, SiluAndMul,
 * down projection; the replicated path when the flag is off).
 *
 *   x          [T x H]    bf16 tokens
 *   w_gate_up  [2I x H]   bf16; rows [0, I) = W_gate, rows [I, 2I) = W_up
 *   w_down     [H x I]    bf16 (out x in)
 *   y          [T x H]    bf16 output, y_capacity >= T*H elements
 *
 *   g = x W_gate^T, u = x W_up^T accumulate in fp32 and are not rounded;
 *   h = bf16_rne(silu(g) * u) is rounded once and kept in the workspace;
 *   y = bf16_rne(h W_down^T) with fp32 accumulation.
 * ------------------------------------------------------------------------- */
MSE_API mse_status mlp_swiglu_forward(const mse_bf16 *x, int64_t T, int64_t H, int64_t I,
                              const mse_bf16 *w_gate_up, const mse_bf16 *w_down,
                              mse_bf16 *y, int64_t y_capacity,
                              void *workspace, size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * Partial outputs of shards [rank_first, rank_first + rank_count) of a tp-way
 * shard of the MLP over the intermediate dimension (prhub analysis of vllm
 * PR #50656, section "关键源码片段": shard r uses gate rows and up rows
 * [r*s, (r+1)*s) and down columns [r*s, (r+1)*s); the down projection is
 * RowParallel and partial over the intermediate dimension per the Kimi-K3 PR,
 * section "Change").  All T tokens are the gathered token set.
 *
 *   partials   [rank_count x T x H], partial_dtype MSE_BF16 or MSE_F32;
 *              partials[i] is the partial of rank rank_first + i, rounded once
 *              from its fp32 accumulator; partials_capacity >= rank_count*T*H.
 *
 * Errors: MSE_ERR_NOT_DIVISIBLE if I % tp or H % tp (the divisibility rule of
 * the sharding gate, prhub section "实现拆解"); MSE_ERR_GEOMETRY if
 * rank_first < 0, rank_count < 1 or rank_first + rank_count > tp.
 * ------------------------------------------------------------------------- */
MSE_API mse_status mlp_swiglu_shard_partial(const mse_bf16 *x, int64_t T, int64_t H, int64_t I,
                                    const mse_bf16 *w_gate_up, const mse_bf16 *w_down,
                                    int tp, int rank_first, int rank_count,
                                    void *partials, mse_dtype partial_dtype,
                                    int64_t partials_capacity,
                                    void *workspace, size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * The partials of shards [rank_first, rank_first + rank_count) summed inside the
 * down projection: a GEMM whose epilogue does the reduce-scatter's sum (Kimi-K3
 * PR, section "Change": the block-end reduce-scatter sums across TP and restores
 * the sequence sharding; prhub analysis of vllm PR #50656, section "关键源码片段":
 * per-shard partials, then stack(partials).sum(0)).  No partial is rounded or
 * stored: the down projection accumulates the group's intermediate columns
 * [rank_first*s, (rank_first + rank_count)*s), s = I/tp, in fp32 (split across
 * CTAs in ascending k order), and the sum is rounded once.
 *
 *   out   [T x H], out_dtype MSE_BF16 or MSE_F32, out_capacity >= T*H.
 *         rank_count = tp: the whole TP group's reduced output; rank r's scatter
 *         share is the row block [r*T/tp, (r+1)*T/tp) (a view; nothing is copied).
 *         rank_count < tp: the group's pre-reduced partial, which a cross-GPU
 *         reduce-scatter would sum with the other groups'.
 *   Same inputs, workspace and stream rules as mlp_swiglu_shard_partial.
 *
 * Errors: MSE_ERR_NOT_DIVISIBLE if I % tp or H % tp; MSE_ERR_GEOMETRY if
 * rank_first < 0, rank_count < 1, rank_first + rank_count > tp or
 * out_capacity < T*H; MSE_ERR_INVALID_ARG for an unknown out_dtype.
 * ------------------------------------------------------------------------- */
MSE_API mse_status mlp_swiglu_shard_forward(const mse_bf16 *x, int64_t T, int64_t H, int64_t I,
                                    const mse_bf16 *w_gate_up, const mse_bf16 *w_down,
                                    int tp, int rank_first, int rank_count,
                                    void *out, mse_dtype out_dtype, int64_t out_capacity,
                                    void *workspace, size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * Whether a dense or shared-expert MLP is to be TP-sharded under sequence
 * parallelism rather than replicated on every rank (prhub analysis of vllm PR
 * #50656, section "实现拆解", item 2; Kimi-K3 PR, sections "Change" and "Trade-off
 * and why it is opt-in"): 1
 * when all of
 *   - enabled: the opt-in switch is on (it is off by default);
 *   - use_sequence_parallel: the model runs with sequence parallelism;
 *   - eligible: the call site may shard (shared experts only on the path whose
 *     MoE block hands them the tokens directly; dense MLPs always);
 *   - tp_size > 1, and hidden_size % tp_size == 0 and
 *     intermediate_size % tp_size == 0;
 * hold, else 0: the MLP stays replicated (the conservative fallback, never an
 * error).  A pure host function: it touches no GPU and needs no device.
 * ------------------------------------------------------------------------- */
MSE_API int mse_shard_sequence_parallel_mlp(int enabled, int use_sequence_parallel, int eligible,
                                            int tp_size, int64_t hidden_size, int64_t intermediate_size);

/* ---------------------------------------------------------------------------
 * Sum of partials: the reduction half of the block-end reduce-scatter
 * (Kimi-K3 PR, section "Change": it sums across TP and restores the sequence
 * sharding).  out[t, n] = bf16_rne( sum_{r ascending} partials[r, t, n] ) with
 * fp32 accumulation.  Rank r's scatter share is the row block
 * [r*T/n_parts, (r+1)*T/n_parts) of `out` (a view; nothing is copied).
 *
 *   partials   [n_parts x T x H] of partial_dtype
 *   out        [T x H] bf16, out_capacity >= T*H
 *
 * Errors: MSE_ERR_NOT_DIVISIBLE if T % n_parts != 0 (token rows cannot be
 * scattered evenly).
 * ------------------------------------------------------------------------- */
MSE_API mse_status shard_sum(const void *partials, mse_dtype partial_dtype, int n_parts,
                     int64_t T, int64_t H, mse_bf16 *out, int64_t out_capacity, void *stream);

/* ---------------------------------------------------------------------------
 * Merged MLA q_a/kv_a latent projection ("[II] TP-shard Kimi MLA latent
 * projections", section "Behavior").  C = q_dim + kv_dim.
 *
 *   x            [T x H] bf16
 *   w            [C x H] bf16, logical row order: q_a rows then kv_a rows
 *   out_logical    nullable, [T x C] bf16 in logical column order [q_a | kv_a]
 *   out_rank_major nullable, [T x C] bf16 in gathered order: for each rank r
 *                  ascending, its q_a columns [r*q/tp, (r+1)*q/tp) then its kv_a
 *                  columns [r*kv/tp, (r+1)*kv/tp)  (the layout a tensor-parallel
 *                  gather of merged column shards produces)
 *   At least one output must be non-null; out_capacity >= T*C.
 *   out = bf16_rne(x w^T) with fp32 accumulation.
 *
 * Errors: MSE_ERR_NOT_DIVISIBLE if q_dim % tp or kv_dim % tp (every merged
 * output size must be divisible by tp, section "Compatibility").
 * ------------------------------------------------------------------------- */
MSE_API mse_status merged_proj_forward(const mse_bf16 *x, int64_t T, int64_t H, const mse_bf16 *w,
                               int64_t q_dim, int64_t kv_dim, int tp,
                               mse_bf16 *out_logical, mse_bf16 *out_rank_major,
                               int64_t out_capacity,
                               void *workspace, size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * Rank-major -> logical reorder alone (MLA page, sections "Behavior" and
 * "Technical reason": the merged-column gather is rank-major and the logical
 * q_a-then-kv_a ranges are restored explicitly).  A pure permutation of 16-bit
 * words: gathered column g = r*(qs+ks) + l maps to logical column
 * r*qs + l (l < qs) or q_dim + r*ks + (l - qs) (l >= qs), qs = q/tp, ks = kv/tp.
 *
 *   rank_major, logical: [T x C] bf16, capacity >= T*C each; must not overlap.
 * ------------------------------------------------------------------------- */
MSE_API mse_status merged_proj_reorder(const mse_bf16 *rank_major, mse_bf16 *logical, int64_t T,
                               int64_t q_dim, int64_t kv_dim, int tp, int64_t capacity,
                               void *stream);

/* ---------------------------------------------------------------------------
 * mlp_swiglu_forward for callers that cannot allocate device memory.  The pages
 * have no counterpart: this is a deployment convenience of this library.
 *
 * Some callers hold only their input and output buffers and have no way to
 * obtain scratch memory: custom-operator interfaces of inference runtimes that
 * pass tensors but no workspace, or code that must not call the CUDA allocator
 * at all (cudaMalloc can synchronise the device and fail under memory pressure).
 * This entry point computes exactly what mlp_swiglu_forward computes, with the
 * same arguments minus the workspace: its scratch (h, split-K partial tiles,
 * tile counters) is a fixed 32 MiB file-scope device array inside the library,
 * which every device that loads the library holds until the process exits.
 *
 *  - Limit: mlp_swiglu_workspace_bytes(T, H, I) <= 32 MiB, e.g. T <= 64 tokens
 *    at hidden 7168 / intermediate 6144.  Larger calls return MSE_ERR_WORKSPACE
 *    and launch nothing.
 *  - It calls no cudaMalloc, cudaFree or allocating library routine.
 *  - The first call on a device performs a one-time set-up on that device
 *    (it looks up the array's device address with cudaGetSymbolAddress); make
 *    that first call before any stream capture.
 *  - Every call on a device shares the one array, and the array keeps the last
 *    call's contents (each call clears the tile counters it needs on `stream`).
 *    Calls whose executions overlap on the GPU (different streams, or several
 *    host threads without ordering) race on the array and give wrong results;
 *    order them on one stream.
 * ------------------------------------------------------------------------- */
MSE_API mse_status mlp_swiglu_forward_static_scratch(const mse_bf16 *x, int64_t T, int64_t H, int64_t I,
                                                     const mse_bf16 *w_gate_up, const mse_bf16 *w_down,
                                                     mse_bf16 *y, int64_t y_capacity, void *stream);

/* ---------------------------------------------------------------------------
 * The replicated SwiGLU MLP with its activations in host memory: the same layer as
 * mlp_swiglu_forward ("[Kimi-K3] Add option to shard the shared expert instead of
 * replicating", section "Change"), for callers whose tokens arrive in, and whose output
 * goes back to, page-locked host memory.
 *
 *   x_host  [T x H] bf16, page-locked host memory mapped into the device's address space
 *           (cudaHostAlloc, or cudaHostRegister with cudaHostRegisterMapped); on systems
 *           whose GPU reaches pageable host memory (cudaDevAttrPageableMemoryAccess, e.g.
 *           Grace-based ones) any host memory
 *   y_host  [T x H] bf16, the same kind of memory, y_capacity >= T*H elements
 *   w_gate_up, w_down  device memory, as for mlp_swiglu_forward
 *   workspace  device memory of mlp_swiglu_host_workspace_bytes(T, H, I) bytes, 256-byte
 *           aligned, zero before first use: 256 bytes of copy counts, two device copies of
 *           x, then the workspace of mlp_swiglu_forward (same rules for reuse)
 *
 * The kernels are launched on `stream` with programmatic dependent launch, so that none of
 * them cuts the overlap of consecutive calls; the down projection writes y straight into
 * y_host.  On the decode-size (swap-AB) kernels the gate_up launch copies x itself: the
 * CTAs that start first (on the SMs the previous layer's down projection leaves free; at
 * most MSE_TUNE_HOST_X_COPIERS) copy one slice each into one of the two device copies, the
 * other one than the previous call on this workspace, and every CTA's token loads wait for
 * all slices.  Elsewhere a copy kernel into the first device copy runs before the layer.
 * x is read while the previous work on the stream still runs, unless x overlaps the y_host
 * of the previous call of this entry point on the same stream (layers chained through host
 * memory), or the previous call on this workspace is unknown (the first, one with another T
 * or H, one on another path, or one captured into a CUDA graph; calls during capture always
 * wait): then it is read once that work is complete.  y_host holds the result once the
 * stream has reached the end of the call (e.g. after cudaStreamSynchronize); the host must
 * not modify x or read y before then.  MSE_ERR_INVALID_ARG if a host pointer is not mapped
 * page-locked memory or the two buffers overlap.
 * ------------------------------------------------------------------------- */
MSE_API size_t mlp_swiglu_host_workspace_bytes(int64_t T, int64_t H, int64_t I);
MSE_API mse_status mlp_swiglu_forward_host(const mse_bf16 *x_host, int64_t T, int64_t H, int64_t I,
                                           const mse_bf16 *w_gate_up, const mse_bf16 *w_down, mse_bf16 *y_host,
                                           int64_t y_capacity, void *workspace, size_t workspace_bytes,
                                           void *stream);

/* ---------------------------------------------------------------------------
 * Errors raised on the device and process-wide settings.
 * ------------------------------------------------------------------------- */

/* Synchronises `stream`, then reads and clears the library's device error word
 * on the current device: MSE_OK, MSE_ERR_TIMEOUT, or MSE_ERR_CUDA if the
 * synchronisation itself failed. */
MSE_API mse_status mse_poll_device_error(void *stream);

/* Upper bound, in nanoseconds, of every device-side wait of later launches
 * (default 2e9 = 2 s).  A wait that runs out sets the device error word, the
 * kernel drains its in-flight copies, frees its tensor memory and returns. */
MSE_API void mse_set_wait_limit_ns(uint64_t ns);
MSE_API uint64_t mse_get_wait_limit_ns(void);

/* Kernel path selection, see mse_kernel_path.  Returns the previous value. */
MSE_API int mse_set_kernel_path(int path);

/* Prefill kernel selection, see mse_prefill_kernel.  Returns the previous value. */
MSE_API int mse_set_prefill_kernel(int kind);

/* Tuning of the decode-size (swap-AB) kernels, process-wide, for later launches.
 *   MSE_TUNE_ISSUE_GROUP  consecutive 64-wide k-blocks per pipeline stage, i.e. each weight row
 *                         is fetched in runs of 128 x value contiguous bytes (1..4); 0 (default)
 *                         = 3 for launches of at most 64 tokens, 2 above
 *   MSE_TUNE_STAGES       shared-memory pipeline depth (0 = as many as fit, default)
 *   MSE_TUNE_CACHE_HINTS  1 = weights evict-first / tokens evict-last in L2 (default), 0 = none
 *   MSE_TUNE_GRID         CTAs of the stream-K grid (at most 160).  0 (default) = chosen per shape:
 *                         among 90-100% of the SMs the count that splits tiles into the fewest
 *                         parts when that is at most three, else one per SM; MLP launches with
 *                         little work (one shard's narrow slice) then at most one CTA per 16
 *                         k-blocks, but not fewer than half of the SMs
 *   MSE_TUNE_SPIN_WAIT    1 = pipeline waits poll (mbarrier.test_wait) instead of suspending
 *   MSE_TUNE_ONE_LAUNCH   decode token counts (T <= 256): 0 = gate_up + SiluAndMul and the down
 *                         projection as two launches (default: with programmatic dependent
 *                         launch this measured fastest); 1 = as passes of one launch, the down
 *                         weights streaming while the last gate_up tiles finish; 2 = one
 *                         launch with the gate_up tiles in two halves, the down pass taking
 *                         the first half's k-blocks first (replicated layer, else as 1)
 *   MSE_TUNE_PDL          1 = kernels are launched with programmatic dependent launch: a kernel
 *                         starts while the previous one in the stream drains and fetches its
 *                         first weight tiles before waiting for it (default); 0 = plain
 *                         stream order
 *   MSE_TUNE_COOP_FINISH  decode token counts: a tile whose reduction is split between at least
 *                         this many CTAs (0..128; 0 = never) is finished jointly by the CTAs for
 *                         which it is the final segment: each waits (bounded) for all parts,
 *                         then sums and writes one slice of the tile's token columns.  Other
 *                         split tiles are finished by the CTA arriving last.  Applies to the
 *                         merged projection and to MLP launches with some tile split this many
 *                         ways (one shard's narrow gate_up slice); same results bit for bit.
 *                         Default 6
 *   MSE_TUNE_PAIR_MIN_T   token counts from which the decode-size kernels run as CTA pairs: one
 *                         256-row weight tile per pair (one M = 256 MMA over both CTAs), each
 *                         CTA holding half of the token rows, so that more weight bytes are in
 *                         flight per SM (0 = never, the default: at 64 and 128 tokens it
 *                         measured no faster than single CTAs)
 *   MSE_TUNE_GRID_DOWN    CTAs of the down-projection swap-AB kernel (0 = as MSE_TUNE_GRID)
 *   MSE_TUNE_CLUSTER_FINISH  1 = when three CTAs of a decode-size kernel cover two tiles exactly
 *                         (gate_up at 64 tokens on 144 CTAs), launch clusters of three and finish
 *                         each two-part tile inside its cluster (same results bit for bit;
 *                         measured within 0.1 us); 0 = through L2 only (default)
 *   MSE_TUNE_L2_PREFETCH  decode token counts: 64-wide k-blocks of weight tiles beyond the
 *                         pipeline that a CTA prefetches into L2 before waiting for the previous
 *                         kernel, if it was not placed on an SM idle at launch: such CTAs start
 *                         while the previous kernel's split-K tail leaves HBM underused.  Applied
 *                         to launches of at most 64 tokens with at least 32 k-blocks per CTA
 *                         (default 8: the decode layer measured 54.2 against 54.35 us with none,
 *                         56.0 with 16; 0 = none)
 *   MSE_TUNE_SWAPAB_MAX_T launches over at least 4096 weight rows (the full layer) take the
 *                         decode-size (swap-AB) kernels up to this token count and the prefill
 *                         kernels above it (0 .. 256, default 160: at 176-256 tokens the full
 *                         layer measured 73 us on the CTA-pair kernel against 80-93 us); narrower
 *                         launches take the swap-AB kernels up to 256 tokens
 *   MSE_TUNE_X_EARLY      1 = mlp_swiglu_forward, mlp_swiglu_shard_partial, mlp_swiglu_shard_forward
 *                         and merged_proj_forward (decode-size kernels) read their x without
 *                         waiting for the previous kernel on the stream when x overlaps neither
 *                         this call's workspace nor anything the previous call on that stream
 *                         writes (its outputs and workspace), the previous call being one of
 *                         these four (independent layers, ranks or requests streamed back to
 *                         back): the first kernel's weight stream then runs during the previous
 *                         call's split-K tail.  Only for callers whose x is not written by a
 *                         kernel of their own that lets its dependents start early
 *                         (programmatic dependent launch) while still writing x.  0 = always
 *                         wait (default).
 *   MSE_TUNE_DOWN_FLAGS   decode token counts, two launches per layer: 1 = the gate_up kernel sets
 *                         a flag per finished 64-column block of h, and each CTA of the down
 *                         kernel, instead of waiting for the gate_up grid to complete, waits
 *                         until the flags of every h block it reads are set (its epilogue still
 *                         waits for the gate_up grid before any store); 0 = off (default)
 *   MSE_TUNE_HOST_X_COPIERS mlp_swiglu_forward_host on the decode-size kernels: the number of
 *                         CTAs of the gate_up launch that copy a slice of x each from host memory
 *                         (the first to start; 1 .. 1024, at most the launch's CTAs; default 16);
 *                         0 = a separate copy kernel before the layer
 *   MSE_TUNE_PAIR_SPLIT   1 = CTA-pair kernel launches of an MLP call at 129-256 tokens with at
 *                         most half as many tiles as clusters split the k-blocks of their tiles
 *                         over more clusters, at most two parts per tile (default); 0 = whole
 *                         tiles only
 * Returns the previous value, or -1 for an unknown key or out-of-range value.
 * Results do not depend on these settings beyond floating-point summation order. */
typedef enum {
    MSE_TUNE_ISSUE_GROUP = 1,
    MSE_TUNE_STAGES = 2,
    MSE_TUNE_CACHE_HINTS = 3,
    MSE_TUNE_GRID = 4,
    MSE_TUNE_SPIN_WAIT = 6,
    MSE_TUNE_ONE_LAUNCH = 7,
    MSE_TUNE_PDL = 8,
    MSE_TUNE_COOP_FINISH = 9,
    MSE_TUNE_PAIR_MIN_T = 10,
    MSE_TUNE_GRID_DOWN = 11,
    MSE_TUNE_CLUSTER_FINISH = 12,
    MSE_TUNE_L2_PREFETCH = 14,
    MSE_TUNE_SWAPAB_MAX_T = 15,
    MSE_TUNE_X_EARLY = 16,
    MSE_TUNE_DOWN_FLAGS = 17,
    MSE_TUNE_HOST_X_COPIERS = 18,
    MSE_TUNE_PAIR_SPLIT = 19
} mse_tune_key;
MSE_API int mse_set_tuning(int key, int value);

/* Launch plan of the decode-size (swap-AB) kernels of an MLP call, computed on the host
 * without a GPU: the CTA counts that mlp_swiglu_forward (tp = 1, rank_count = 1) or a
 * group of rank_count consecutive ranks of a tp-way split (mlp_swiglu_shard_partial /
 * mlp_swiglu_shard_forward, slices of I / tp intermediate columns; pages P1 "Change",
 * P2 "关键源码片段") would launch for T tokens on a device with sm_count SMs, with the
 * tuning keys as currently set; x_early = 1 when the call's early token loads apply (a
 * streamed call whose x the previous call does not write, MSE_TUNE_X_EARLY).
 * out[8] (host memory, written): [0] 1 when the call takes the swap-AB kernels, 0 when it
 * takes the prefill or the generic kernels (shapes off the 64-column grid, or
 * mse_set_kernel_path(MSE_PATH_GENERIC); then [1..7] are 0); [1] gate_up CTAs; [2] down
 * CTAs; [3] / [4] the largest number of CTAs a gate_up / down tile is split between;
 * [5] token tile width (T rounded up to 16); [6] k-blocks per pipeline stage; [7] stages.
 * Returns MSE_OK; MSE_ERR_INVALID_ARG (null out, non-positive size, rank_count outside
 * [1, tp]); MSE_ERR_NOT_DIVISIBLE (I by tp); MSE_ERR_UNSUPPORTED_SHAPE when a tuning key
 * makes the shape depend on the device's occupancy (MSE_TUNE_ONE_LAUNCH,
 * MSE_TUNE_PAIR_MIN_T, MSE_TUNE_CLUSTER_FINISH). */
MSE_API int mse_mlp_launch_plan(int64_t T, int64_t H, int64_t I, int tp, int rank_count, int x_early,
                                int sm_count, int32_t *out);

/* The same for merged_proj_forward (page P4 "Behavior": the 2112 x 7168 merged q_a / kv_a
 * projection).  out[8]: [0] 1 when the call takes the swap-AB kernel (0: the prefill or the
 * generic kernels, then [1..7] are 0); [1] CTAs; [2] the largest number of CTAs a 128-row
 * weight tile is split between; [3] 1 when the tiles' parts are finished jointly (every part's
 * CTA sums a slice of the token columns, MSE_TUNE_COOP_FINISH); [4] token tile width;
 * [5] k-blocks per pipeline stage; [6] stages; [7] 0.  Errors as mse_mlp_launch_plan (q_dim
 * and kv_dim by tp for MSE_ERR_NOT_DIVISIBLE). */
MSE_API int mse_merged_launch_plan(int64_t T, int64_t H, int64_t q_dim, int64_t kv_dim, int tp, int sm_count,
                                   int32_t *out);

/* Failure-detection self test: launches one CTA that waits on a barrier no one
 * arrives on, bounded by `limit_ns`.  The wait runs out by design; the kernel
 * records MSE_ERR_TIMEOUT in the device error word and returns, leaving the
 * context usable.  Read the result with mse_poll_device_error(). */
MSE_API mse_status mse_selftest_wait_timeout(uint64_t limit_ns, void *stream);

/* Timing hook for profiling harnesses.  While set, every mlp_swiglu_forward,
 * mlp_swiglu_shard_partial and mlp_swiglu_shard_forward call on the tensor-core
 * path records ev_begin before its first kernel, ev_mid between the gate_up and
 * the down kernel, and ev_end after the down kernel, on its stream (cudaEvent_t
 * handles passed as void*; all three non-null, or all null to clear).  The
 * records separate the two kernels, so launches made while the hook is set do
 * not overlap them. Process-wide; not meant for concurrent callers. */
MSE_API void mse_set_phase_events(void *ev_begin, void *ev_mid, void *ev_end);

/* ---------------------------------------------------------------------------
 * The routed experts beside the shared expert: routing, products in 8 bits with a
 * scale for each block of 128, and the experts' layer.  Inference only, like the
 * rest of the library.
 *
 * Sizes beyond these are MSE_ERR_INVALID_ARG: token rows (T, rows; T * top_k of the experts) 2^30; weight rows and
 * inner sizes (N, K, H, I) 2^22; row pitches 2^32 elements; blocks of 128 x 128 of one fp8_block_quantise 2^31 - 1.
 * ------------------------------------------------------------------------- */

typedef enum { MSE_SCORE_SOFTMAX = 0, MSE_SCORE_SIGMOID = 1 } mse_score;

/* Limits of moe_route: experts, groups, chosen experts per token. */
#define MSE_ROUTE_MAX_EXPERTS 1024
#define MSE_ROUTE_MAX_GROUPS 32
#define MSE_ROUTE_MAX_TOP_K 32

/* Routing of T tokens to E experts.
 *
 *   logits   [T x E]      bf16 or fp32 (logits_dtype), row pitch ld >= E elements
 *   bias     [E]          fp32 for the choice alone, or null
 *   ids      [T x top_k]  int32: the chosen experts, best first; -1 where no expert is left
 *   weights  [T x top_k]  fp32, 0 where ids is -1; capacity >= T*top_k elements of each
 *
 * An expert is open to a token when its logit is above the lowest finite bf16 value; -inf,
 * either type's lowest value and NaN close it.  In fp32:
 *   score  = 1 / (1 + e^-l), or e^(l - max) / sum over the open experts (softmax; the sum
 *            as if rounded once, so that no choice depends on an order of summation);
 *   choice = score + bias (an expert whose choice is NaN or -inf is not chosen, and counts for nothing in its group);
 *   groups: experts [g E / n_group, (g + 1) E / n_group); a group's value is the sum of its
 *            group_top (1 or 2) best open choices (of fewer where fewer are open), and only
 *            the topk_group best groups stay open;
 *   ids    = the top_k best open choices; equal ones go to the lower index, groups too;
 *   weight = score of the chosen (without the bias), divided by their sum if renormalise
 *            (by nothing where that sum is 0), times scale.
 * A token with no open expert gets ids -1 and weights 0.  A logit of +inf makes every softmax score of
 * its token NaN: equal choices, so the lowest open experts (of the lowest topk_group groups with one),
 * with weights NaN.
 * MSE_ERR_INVALID_ARG: null pointer, non-positive size, bad enum, ld < E, E, n_group or top_k
 * beyond the limits, topk_group outside [1, n_group], top_k above the topk_group * E / n_group
 * experts that stay, group_top not 1 or 2; MSE_ERR_NOT_DIVISIBLE: E by n_group;
 * MSE_ERR_GEOMETRY: capacity. */
MSE_API mse_status moe_route(const void *logits, mse_dtype logits_dtype, int64_t T, int64_t E, int64_t ld,
                             const float *bias, mse_score scoring, int n_group, int topk_group, int group_top,
                             int top_k, int renormalise, float scale, int32_t *ids, float *weights,
                             int64_t capacity, void *stream);

/* Rounding to 8 bits (e4m3: 4 exponent bits, 3 fraction bits, largest 448) with one scale for
 * each block of block_rows x 128 (block_rows 1: activations; 128: weights):
 *   a = max(max |B|, 2^-100),   scale = a / 448,   q = e4m3(448 B / a) to nearest, ties to even.
 * A block that holds an infinity or a NaN stands for NaN throughout.
 *   x       [rows x K]  bf16, row pitch ldx >= K
 *   q       [rows x K]  row pitch ldq >= K bytes, q_capacity >= (rows - 1) * ldq + K
 *   scales  [ceil(rows / block_rows) x ceil(K / 128)] fp32, scales_capacity elements */
MSE_API mse_status fp8_block_quantise(const mse_bf16 *x, int64_t rows, int64_t K, int64_t ldx, int block_rows,
                                      uint8_t *q, int64_t ldq, int64_t q_capacity, float *scales,
                                      int64_t scales_capacity, void *stream);

/* out [T x N] = sum over k-blocks b of xs[t, b] ws[n / 128, b] sum_{k in b} xq[t, k] wq[n, k].
 *   xq [T x K] e4m3, row pitch ldx >= K bytes;  xs [T x ceil(K / 128)] fp32
 *   wq [N x K] e4m3, row pitch ldw >= K bytes;  ws [ceil(N / 128) x ceil(K / 128)] fp32
 *   out bf16 or fp32 (out_dtype), out_capacity >= T*N elements
 * Each block's products are summed on the tensor cores and added, scaled, to an fp32 sum; out is
 * rounded once.  The tensor-core kernels take row pitches that are multiples of 16 with 16-byte
 * aligned operands; anything else takes the generic kernels. */
MSE_API mse_status fp8_block_matmul(const uint8_t *xq, int64_t ldx, const float *xs, const uint8_t *wq, int64_t ldw,
                                    const float *ws, int64_t T, int64_t N, int64_t K, void *out,
                                    mse_dtype out_dtype, int64_t out_capacity, void *stream);

/* Workspace of fp8_block_linear for every token count up to T (0 on invalid arguments):
 * 256-byte aligned, need not be zeroed, holds x in 8 bits. */
MSE_API size_t fp8_block_linear_workspace_bytes(int64_t T, int64_t N, int64_t K);

/* fp8_block_quantise of x [T x K] bf16 (row pitch ldx) in blocks of 1 x 128, then
 * fp8_block_matmul, in one call.  y may lie over x. */
MSE_API mse_status fp8_block_linear(const mse_bf16 *x, int64_t ldx, const uint8_t *wq, int64_t ldw, const float *ws,
                                    int64_t T, int64_t N, int64_t K, void *y, mse_dtype y_dtype, int64_t y_capacity,
                                    void *workspace, size_t workspace_bytes, void *stream);

/* Workspace of moe_experts_forward for every token count up to T with the same or smaller other
 * sizes (0 on invalid arguments): 256-byte aligned, need not be zeroed. */
MSE_API size_t moe_experts_workspace_bytes(int64_t T, int top_k, int64_t E, int64_t H, int64_t I);

/* The routed experts of a rank that holds experts [first_expert, first_expert + E):
 *
 *   y[t] = shared[t] + sum_j weights[t, j] * W_down,e h,   e = ids[t, j] - first_expert,
 *   [g; u] = W_gate_up,e x[t],   h = silu(g) * u,
 *
 * over the j whose e lies in [0, E) (others, -1 among them, belong to other ranks or to nobody).
 * x and h are rounded to e4m3 in blocks of 1 x 128; products as in fp8_block_matmul; the sum over
 * j runs in fp32, ascending, on top of shared, and is rounded once.
 *
 *   x         [T x H]         bf16
 *   ids       [T x top_k]     int32;   weights [T x top_k] fp32
 *   w_gate_up [E x 2I x H]    e4m3, row pitch ld_gate_up >= H; rows [0, I) gate, [I, 2I) up
 *   s_gate_up [E x 2 ceil(I / 128) x ceil(H / 128)] fp32; gate's blocks, then up's, each half's
 *                             blocks counted from its own first row
 *   w_down    [E x H x I]     e4m3, row pitch ld_down >= I
 *   s_down    [E x ceil(H / 128) x ceil(I / 128)] fp32
 *   shared    [T x H]         bf16, or null for 0
 *   y         [T x H]         bf16, y_capacity >= T*H elements (x or shared itself is allowed)
 * top_k <= MSE_ROUTE_MAX_TOP_K, E <= MSE_ROUTE_MAX_EXPERTS; T * top_k <= 2^30. */
MSE_API mse_status moe_experts_forward(const mse_bf16 *x, int64_t T, int64_t H, const int32_t *ids,
                                       const float *weights, int top_k, const uint8_t *w_gate_up, int64_t ld_gate_up,
                                       const float *s_gate_up, const uint8_t *w_down, int64_t ld_down,
                                       const float *s_down, int64_t E, int64_t I, int64_t first_expert,
                                       const mse_bf16 *shared, mse_bf16 *y, int64_t y_capacity, void *workspace,
                                       size_t workspace_bytes, void *stream);

/* The kernels that fp8_block_matmul and fp8_block_linear would launch for operands with 16-byte rows, on the current
 * device.  out[4] (host memory, written): [0] token rows of a tile, 16, 32 or 64 (weights on the MMA's 128-row side) or 256
 * (CTA pairs), 0 when the generic kernels are forced (then [1..3] are 0); [1] CTAs, or pairs, that share a tile's
 * k-blocks; [2] CTAs; [3] 1 when fp8_block_linear rounds its tokens inside the product's kernel (y apart from x).
 * MSE_ERR_INVALID_ARG as the calls; MSE_ERR_UNSUPPORTED_DEVICE without a device. */
MSE_API mse_status mse_fp8_launch_plan(int64_t T, int64_t N, int64_t K, int32_t *out);

/* The same for moe_experts_forward: out[8]: [0] token rows of a tile, 16, 32 or 256 (0: generic kernels, then [1..5] are
 * 0); [1] / [2] gate_up's CTAs to a tile's k-blocks and CTAs; [3] / [4] down's; [5] 1 when gate_up finds its tiles in the
 * ids; [6] 1 when the ids are counted by kernels of their own; [7] 0. */
MSE_API mse_status mse_moe_launch_plan(int64_t T, int top_k, int64_t E, int64_t H, int64_t I, int32_t *out);

/* ---------------------------------------------------------------------------
 * Tokens sorted by expert and back with their weights, with the gradients of both ways, for experts that the
 * caller runs (any product over rows [offsets[e], offsets[e + 1])).
 *
 * Sizes beyond these are MSE_ERR_INVALID_ARG: T, rows and T * top_k 2^30; H 2^22; row pitches 2^32 values; top_k and E
 * MSE_ROUTE_MAX_TOP_K and MSE_ROUTE_MAX_EXPERTS.  Outputs and workspaces lie apart from the inputs and from each other, but for
 * those named (of rows with a pitch, all from the first value to the last counts): else MSE_ERR_INVALID_ARG.  Calls that run at
 * the same time need workspaces of their own, graphs among them.
 * ------------------------------------------------------------------------- */

/* Workspace of moe_sort for every token count up to T (0 on invalid arguments): 256-byte aligned, need not be zeroed. */
MSE_API size_t moe_sort_workspace_bytes(int64_t T, int top_k, int64_t E);

/* The rows of a rank that holds experts [first_expert, first_expert + E), sorted by expert, in the order of t * top_k + j
 * within each:
 *
 *   rows[place[t, j]] = x[t]  for every pair (t, j) with ids[t, j] - first_expert in [0, E); place is -1 for the others
 *   offsets[e] = the first row of expert e; offsets[E] = the rows in all
 *
 *   x           [T x H]          values of value_bytes 1, 2 or 4 (copied as they are), row pitch ldx >= H
 *   ids         [T x top_k]      int32, as moe_route gives them
 *   scales      [T]              fp32 for each token, copied along to row_scales [T * top_k]; or null, both
 *   rows        [T * top_k x H]  row pitch ldr >= H, rows_capacity >= (T * top_k - 1) * ldr + H; rows from offsets[E] on are
 *                                left as they were, and the values between H and ldr too
 *   place       [T x top_k]      int32;   offsets [E + 1] int32
 * MSE_ERR_GEOMETRY: rows_capacity. */
MSE_API mse_status moe_sort(const void *x, int value_bytes, int64_t T, int64_t H, int64_t ldx, const int32_t *ids, int top_k,
                            int64_t E, int64_t first_expert, const float *scales, void *rows, int64_t ldr,
                            int64_t rows_capacity, float *row_scales, int32_t *place, int32_t *offsets, void *workspace,
                            size_t workspace_bytes, void *stream);

/* y[t] = base[t] + sum_j weights[t, j] rows[place[t, j]], in fp32, ascending j, rounded once.  Pairs whose place is not in
 * [0, n_rows) add nothing.
 *   rows     [n_rows x H]  bf16 or fp32, row pitch ldr >= H;   place [T x top_k] int32
 *   weights  [T x top_k]   fp32, or null for 1
 *   base     [T x H]       of y's type (y itself is allowed), or null for 0
 *   y        [T x H]       bf16 or fp32, y_capacity >= T*H elements
 * With the gradient of sorted rows as rows and no weights: the gradient of moe_sort, dx[t] = sum_j drows[place[t, j]]. */
MSE_API mse_status moe_unsort(const void *rows, mse_dtype rows_dtype, int64_t n_rows, int64_t ldr, const int32_t *place,
                              const float *weights, int64_t T, int64_t H, int top_k, const void *base, void *y,
                              mse_dtype y_dtype, int64_t y_capacity, void *stream);

/* The gradients of moe_unsort from dy [T x H] (bf16 or fp32):
 *   drows[place[t, j]] = weights[t, j] dy[t],    dweights[t, j] = <rows[place[t, j]], dy[t]> in fp32
 * (base's is dy).  Pairs whose place is not in [0, n_rows) have dweights 0.
 *   weights   [T x top_k]   fp32, or null for 1 (then dweights is null, and rows is not read)
 *   rows      [n_rows x H]  as moe_unsort had them, row pitch ldr >= H
 *   drows     [n_rows x H]  of rows' type (rows itself, with its pitch, is allowed), row pitch ldd >= H, drows_capacity >=
 *                           (n_rows - 1) * ldd + H; rows that are no pair's place are left as they were
 *   dweights  [T x top_k]   fp32 (weights itself is allowed)
 * place holds no row twice, as moe_sort gives it (else that row of drows is either pair's). */
MSE_API mse_status moe_unsort_backward(const void *dy, mse_dtype dy_dtype, const int32_t *place, const float *weights,
                                       const void *rows, mse_dtype rows_dtype, int64_t ldr, int64_t n_rows, int64_t T,
                                       int64_t H, int top_k, void *drows, int64_t ldd, int64_t drows_capacity,
                                       float *dweights, void *stream);

/* ---------------------------------------------------------------------------
 * Products in 8-bit integers: a scale for each row of either operand (each token, each output channel).
 *
 * Sizes beyond these are MSE_ERR_INVALID_ARG: T, rows and groups * N 2^30; N 2^22; K 2^17 - 1 (so that a sum fits 32 bits;
 * int8_quantise 2^22); groups MSE_ROUTE_MAX_EXPERTS; row pitches 2^32 values.  So are outputs and workspaces that lie over an
 * input or over each other (of rows with a pitch, all from the first value to the last counts), but for y over x in int8_linear.
 * ------------------------------------------------------------------------- */

/* Rows rounded to 8-bit integers:  a = max(max |r|, 2^-100),  scale = a / 127,  q = rint(127 r / a), ties to even, of a
 * quotient in fp32.  r = x, or with swiglu silu(x[.., :K]) * x[.., K:], silu(g) = g / (1 + e^-g), in fp32 (0 where e^-g is beyond
 * it, g < -88.7).  A row with an infinity or a NaN stands for NaN throughout (scale NaN, q 0).
 *   x       [rows x K], swiglu: [rows x 2K]  bf16 or fp32, row pitch ldx
 *   last    null, or one int32 on the device: rows from *last on are left alone (offsets + E of moe_sort)
 *   q       [rows x K]  int8, row pitch ldq >= K, q_capacity >= (rows - 1) * ldq + K
 *   scales  [rows] fp32 */
MSE_API mse_status int8_quantise(const void *x, mse_dtype x_dtype, int64_t rows, int64_t K, int64_t ldx, int swiglu,
                                 const int32_t *last, int8_t *q, int64_t ldq, int64_t q_capacity, float *scales,
                                 void *stream);

/* Workspace of the products for every token count up to T with the same or smaller other sizes (0 on invalid arguments):
 * 256-byte aligned, need not be zeroed.  Calls that run at the same time need workspaces of their own, graphs among them. */
MSE_API size_t int8_workspace_bytes(int64_t T, int64_t N, int64_t K, int64_t groups);

/* out[t, n] = (sum_k xq[t, k] wq[n, k]) xs[t] ws[n]: the sum is the integer itself, whatever the kernel; it is rounded to
 * fp32, multiplied by xs[t], then by ws[n], and rounded to out's type.
 *   xq [T x K] int8, row pitch ldx >= K;  xs [T] fp32
 *   wq [N x K] int8, row pitch ldw >= K;  ws [N] fp32
 *   out [T x N] bf16 or fp32, out_capacity >= T*N elements
 * The tensor-core kernels, and those for few rows on every path but MSE_PATH_GENERIC, take row pitches of wq that are
 * multiples of 16 and a 16-byte aligned wq; anything else takes the generic kernels. */
MSE_API mse_status int8_matmul(const int8_t *xq, int64_t ldx, const float *xs, const int8_t *wq, int64_t ldw, const float *ws,
                               int64_t T, int64_t N, int64_t K, void *out, mse_dtype out_dtype, int64_t out_capacity,
                               void *workspace, size_t workspace_bytes, void *stream);

/* The same of sorted rows with their group's weights: rows [offsets[g], offsets[g + 1]) of xq with wq[g] [N x K] and ws[g]
 * [N].  offsets [groups + 1] int32 ascends, as moe_sort gives it (else which rows are written is open); rows of out outside
 * them are left as they were.  T: rows of xq and out (offsets beyond count as T).  The kernel is chosen for T rows: of rows of
 * which many belong to no group, those that do may be passed alone, with fewer as T (their number has to be on the host then). */
MSE_API mse_status int8_grouped_matmul(const int8_t *xq, int64_t ldx, const float *xs, const int32_t *offsets, int64_t groups,
                                       const int8_t *wq, int64_t ldw, const float *ws, int64_t T, int64_t N, int64_t K,
                                       void *out, mse_dtype out_dtype, int64_t out_capacity, void *workspace,
                                       size_t workspace_bytes, void *stream);

/* The kernels that int8_matmul and int8_linear (groups 0), or int8_grouped_matmul, would launch for weights with 16-byte rows, on
 * the current device.  out[4] (host memory, written): [0] token rows of a tile: 1, 2 or 4 (CUDA cores), 16, 32 or 64 (tensor
 * cores, weights on the MMA's 128-row side) or 256 (CTA pairs), 0 when the generic kernels are forced (then [1] and [2] are 0);
 * [1] CTAs, or pairs, that share a tile's k-blocks; [2] 1 when int8_linear rounds its token inside the product's kernel (y apart
 * from x); [3] 0.  MSE_ERR_INVALID_ARG as the calls; MSE_ERR_UNSUPPORTED_DEVICE without a device. */
MSE_API mse_status mse_int8_launch_plan(int64_t T, int64_t N, int64_t K, int64_t groups, int32_t *out);

/* int8_quantise of x [T x K] (bf16 or fp32, row pitch ldx), then int8_matmul, in one call.  y may lie over x. */
MSE_API mse_status int8_linear(const void *x, mse_dtype x_dtype, int64_t ldx, const int8_t *wq, int64_t ldw, const float *ws,
                               int64_t T, int64_t N, int64_t K, void *y, mse_dtype y_dtype, int64_t y_capacity,
                               void *workspace, size_t workspace_bytes, void *stream);

/* Human-readable name of a status code (static string). */
MSE_API const char *mse_status_string(mse_status s);

/* Library version string, e.g. "mse 0.1 sm_103a". */
MSE_API const char *mse_version(void);

#ifdef __cplusplus
}
#endif
#endif /* MSE_H */
