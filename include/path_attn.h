/*
 * path_attn.h — C ABI of the GB300 (sm_103a) PaTH attention library.
 *
 * PaTH attention (Yang et al., "PaTH Attention: Position Encoding via Accumulating Householder
 * Transformations", arXiv 2505.16381v2; reading notes at cc.laoqi.cc/papers/2505.16381/v2/r1):
 *
 *   H_t        = I - beta_t w_t w_t^T                          (notes §2.1)
 *   logit(i,j) = scale * k_j^T H_{j+1} H_{j+2} ... H_i q_i       (j <= i; H_j excluded, H_i included)
 *              + sum_{s=j+1..i} log f_s                         (optional PaTH-FoX gate, notes §2.5)
 *   o_i        = sum_{j<=i} softmax_j(logit(i,.)) v_j,  lse_i = log sum_{j<=i} exp(logit(i,j))
 *
 * Conventions shared by every entry point
 * ----------------------------------------
 *  - All tensor arguments are DEVICE pointers into memory the caller owns (cudaMalloc, PyTorch,
 *    ...).  The library allocates nothing, frees nothing, and keeps no state between calls
 *    other than a per-device attribute cache.  Calls are reentrant.
 *  - Layouts are dense row-major: q,k,v,w,o,dO,dq,dk,dv,dw are [batch][heads][seqlen][head_dim];
 *    beta, log_f, lse, dbeta are [batch][heads][seqlen].  Decode vectors are
 *    [batch][heads][head_dim], beta_t is [batch][heads], caches are
 *    [batch][heads][capacity][head_dim].
 *  - Element type of q,k,v,w,o,dO,dq,dk,dv,dw and of the caches: the descriptor's dtype
 *    (PATH_BF16 or PATH_FP32).  beta, log_f, lse, dbeta are always float32.  Arithmetic
 *    accumulates in fp32.
 *  - Every tensor pointer must be 16-byte aligned.  Workspace ("ws") pointers must be 256-byte
 *    aligned and hold at least the size returned by the matching *_workspace_size function.
 *  - beta is clamped to [0, 2] inside the kernels (the range of the 2*sigmoid parameterisation,
 *    notes §2.1/§2.2).  Inputs already in range are used unchanged; dbeta is the gradient with
 *    respect to the clamped value.  w is used as given (it is not renormalised).
 *  - "stream" is a cudaStream_t passed as void* (NULL = legacy default stream).  Work is
 *    enqueued asynchronously; faults inside kernels surface at the caller's next sync, and a
 *    tensor-core kernel whose internal wait gave up is reported by path_attn_workspace_status.
 *  - Errors: every argument is validated before any CUDA call; on a validation error nothing
 *    is launched and a status below is returned.  Launch failures return PATH_ERR_CUDA.
 *    No exception crosses the ABI.
 */
#ifndef PATH_ATTN_H
#define PATH_ATTN_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PATH_OK = 0,
  PATH_ERR_INVALID_ARG = 1,  /* null pointer, non-positive size, misaligned pointer, bad enum */
  PATH_ERR_UNSUPPORTED = 2,  /* valid but not implemented (head_dim not 64 or 128, chunk value, ...) */
  PATH_ERR_WORKSPACE = 3,    /* ws_bytes smaller than the required workspace */
  PATH_ERR_CAPACITY = 4,     /* decode: t + 1 > capacity */
  PATH_ERR_CUDA = 5,         /* a CUDA runtime call or kernel launch failed */
  PATH_ERR_INTERNAL = 6
} path_status_t;

typedef enum { PATH_BF16 = 0, PATH_FP32 = 1 } path_dtype_t;

typedef struct {
  int batch;      /* > 0 */
  int heads;      /* > 0 */
  int seqlen;     /* L > 0 */
  int head_dim;   /* d: 64 or 128.  bf16 at 64 runs the tcgen05 kernels (chunk 64); the bf16
                     forward at 128 runs the head-dim-128 tcgen05 kernels (chunk 0 or 64: 64-row
                     chunks); fp32 and the backward at 128 run the fp32 CUDA-core kernels with
                     32-row chunks (fp32 chunk 64 at 128 is PATH_ERR_UNSUPPORTED) */
  int dtype;      /* path_dtype_t of q,k,v,w,o (and dO,dq,dk,dv,dw in the backward) */
  float scale;    /* multiplies the Householder-path logit; the forget bias is added unscaled */
  int chunk;      /* UT chunk size B; 0 lets the library choose (see path_attn_chunk) */
} path_attn_desc_t;

typedef struct {
  int batch;       /* > 0 */
  int heads;       /* > 0 */
  int head_dim;    /* 64 or 128 (path_decode_step_noalloc: 64 only) */
  int capacity;    /* rows allocated per (batch, head) in each cache */
  int cache_dtype; /* path_dtype_t of the caches and of q_t,k_t,v_t,w_t,o_t */
  float scale;     /* logit multiplier */
} path_decode_desc_t;

/* Human-readable name of a status code (static string, never NULL). */
const char* path_status_string(int status);

/* Chunk size B used by the forward (for_backward = 0) or backward (1) pass for this
 * descriptor, or minus a path_status_t if the descriptor is invalid/unsupported. Host only. */
int path_attn_chunk(const path_attn_desc_t* desc, int for_backward);

/* Bytes of workspace path_attn_fwd (for_backward = 0) or path_attn_bwd (for_backward = 1)
 * needs for this descriptor; 0 if the descriptor is invalid.  Host only, no CUDA call. */
size_t path_attn_workspace_size(const path_attn_desc_t* desc, int for_backward);

/*
 * Forward pass: o and lse for every (batch, head, row).
 *
 * Steps (notes §2.6–§2.7): per chunk of B positions, the UT transform
 * U = (I + strictLower(D W W^T))^{-1} D by forward substitution; the boundary-adjusted queries
 * Q<- = Q - lower(Q W^T) U W, keys K-> = K - (U strictLower(W K^T))^T W and chunk transform
 * F = I - W^T U^T W; the diagonal chunk from lower(Q K^T) - lower(Q W^T) U strictLower(W K^T);
 * then, per query chunk, a right-to-left scan over earlier chunks (scores Z K->^T, online
 * softmax, O += P V, Z <- Z F^T).
 *
 * log_f: forget-gate log values (<= 0) or NULL for plain PaTH.
 * o: output, desc dtype.  lse: float32 natural-log log-sum-exp per row (the backward needs it).
 * ws/ws_bytes: scratch of at least path_attn_workspace_size(desc, 0) bytes; its contents on
 * entry are ignored and on exit are unspecified.
 */
int path_attn_fwd(const path_attn_desc_t* desc, const void* q, const void* k, const void* v,
                  const void* w, const float* beta, const float* log_f, void* o, float* lse,
                  void* ws, size_t ws_bytes, void* stream);

/*
 * Backward pass: gradients of sum(dO * o) with respect to q, k, v, w and beta, given the
 * forward's o and lse for the same inputs.  The pages give no backward; this is the exact
 * derivative of the forward definition, evaluated blockwise: recomputed per-chunk UT
 * quantities, a descending scan that stores the transported queries Z_c, an ascending adjoint
 * scan G_c = dS_c K->_c + G_{c-1} F_c with dF_c += G_{c-1}^T Z_c, then the chain rule through
 * the per-chunk UT quantities.
 *
 * dq,dk,dv,dw: desc dtype outputs (overwritten).  dbeta: float32 (overwritten).
 * PaTH-FoX (forget gate, notes §2.5): pass the forward's log_f; dlog_f (float32, same shape,
 * may be NULL) receives dL/dlog f.  dlog_f without log_f is PATH_ERR_INVALID_ARG.  Both paths
 * take the forget gate; the bf16 tensor-core path recovers the logit gradient from the scaled
 * one, so there log_f with scale == 0 returns PATH_ERR_UNSUPPORTED (the fp32 path accepts it).
 * ws: at least path_attn_workspace_size(desc, 1) bytes.
 */
int path_attn_bwd(const path_attn_desc_t* desc, const void* q, const void* k, const void* v,
                  const void* w, const float* beta, const float* log_f, const void* o,
                  const float* lse, const void* dO, void* dq, void* dk, void* dv, void* dw,
                  float* dbeta, float* dlog_f, void* ws, size_t ws_bytes, void* stream);

/*
 * The same two passes split into their phases, so that a caller can time or overlap them.
 * path_attn_fwd(...) is path_attn_fwd_phases(PATH_FWD_ALL, ...); path_attn_bwd likewise.
 * Phases must run in the listed order on one stream with the same arguments and the same
 * workspace, and nothing else may use that workspace in between.  Arguments, validation and
 * errors are those of the full call (every pointer is checked whatever the phase);
 * phases == 0 or an unknown bit gives PATH_ERR_INVALID_ARG.
 *   forward:  PREPARE = per-chunk UT transform, Q<-, K->, F and diagonal-chunk softmax state
 *             into ws;  SCAN = right-to-left chunk scan writing o and lse.
 *   backward: PREPARE = zero the accumulators, D_i = dO_i . o_i, recompute the per-chunk UT
 *             quantities;  SCAN = descending Z pass and ascending adjoint scan (accumulates
 *             dV, dK->, dF, writes dQ<- in ws);  FINISH = diagonal-chunk and UT backward
 *             writing dq, dk, dv, dw, dbeta.
 */
enum { PATH_FWD_PREPARE = 1, PATH_FWD_SCAN = 2, PATH_FWD_ALL = 3 };
enum { PATH_BWD_PREPARE = 1, PATH_BWD_SCAN = 2, PATH_BWD_FINISH = 4, PATH_BWD_ALL = 7 };
/* Optional bit for path_attn_bwd_phases(PREPARE): the workspace already holds the forward's
 * per-chunk preparation for exactly these inputs and descriptor, because path_attn_fwd was run
 * with this same workspace (sized by path_attn_workspace_size(desc, 1)) and nothing used it since.
 * PREPARE then skips recomputing it (the bf16 tensor-core path; ignored by the fp32 path).  If the
 * statement is false the gradients are wrong; nothing detects it. */
enum { PATH_BWD_REUSE_FWD = 8 };
/* Optional bit for path_attn_fwd_phases(SCAN), for a forward that a backward will follow (a
 * training step): ws must be backward-sized (path_attn_workspace_size(desc, 1), else
 * PATH_ERR_WORKSPACE), and the scan also stores every transported query tile Z_n (§2.7: the
 * queries carried across earlier chunks) in ws, which the backward needs.  The bf16
 * tensor-core path at head_dim 64 only; ignored otherwise. */
enum { PATH_FWD_STORE_Z = 4 };
/* Optional bit for path_attn_bwd_phases(PREPARE): the workspace already holds the transported
 * query tiles because the forward ran with PATH_FWD_STORE_Z on it (same inputs, descriptor and
 * workspace, nothing used it since); PREPARE then skips recomputing them.  Same caveat and scope
 * as PATH_BWD_REUSE_FWD. */
enum { PATH_BWD_Z_FROM_FWD = 16 };

int path_attn_fwd_phases(int phases, const path_attn_desc_t* desc, const void* q, const void* k,
                         const void* v, const void* w, const float* beta, const float* log_f,
                         void* o, float* lse, void* ws, size_t ws_bytes, void* stream);

int path_attn_bwd_phases(int phases, const path_attn_desc_t* desc, const void* q, const void* k,
                         const void* v, const void* w, const float* beta, const float* log_f,
                         const void* o, const float* lse, const void* dO, void* dq, void* dk,
                         void* dv, void* dw, float* dbeta, float* dlog_f, void* ws,
                         size_t ws_bytes, void* stream);

/* Bytes of workspace path_decode_step needs for any t < capacity; 0 if invalid. Host only. */
size_t path_decode_workspace_size(const path_decode_desc_t* desc);

/*
 * One decode step at position t (notes §2.8, Eq. (1)).  On entry rows 0..t-1 of each cache
 * hold the keys/values of earlier positions, keys already transported to position t-1.
 * The step
 *   1. rewrites every cached key in place: k_j <- k_j - beta_t (w_t . k_j) w_t   (j < t),
 *   2. appends k_t and v_t unchanged at row t,
 *   3. writes o_t = sum_j softmax_j(scale k_j . q_t) v_j over j = 0..t.
 * Requires 0 <= t and t + 1 <= capacity (else PATH_ERR_CAPACITY).
 * q_t,k_t,v_t,w_t,o_t: [batch][heads][head_dim] in cache_dtype; beta_t: [batch][heads] float32.
 * ws: at least path_decode_workspace_size(desc) bytes (per-split partial softmax states).
 */
int path_decode_step(const path_decode_desc_t* desc, void* k_cache, void* v_cache, int t,
                     const void* q_t, const void* k_t, const void* v_t, const void* w_t,
                     const float* beta_t, void* o_t, void* ws, size_t ws_bytes, void* stream);

/* Bytes of workspace path_decode_prefill needs for a prompt of prompt_len tokens (the fp32
 * chunk transforms of the prompt); 0 if the descriptor or prompt_len is invalid. Host only. */
size_t path_decode_prefill_workspace_size(const path_decode_desc_t* desc, int prompt_len);

/*
 * Prefill -> decode hand-off (notes §2.8, last paragraph: after a prefill every key must be
 * aligned to the prompt end, by the block suffix products).  Fills rows 0..prompt_len-1 of each
 * cache so that path_decode_step can continue at t = prompt_len:
 *   k_cache row j = H_{L-1} ... H_{j+1} k_j   (H_t = I - beta_t w_t w_t^T, L = prompt_len),
 *   v_cache row j = v_j,
 * i.e. exactly what prompt_len calls of path_decode_step from an empty cache would leave there.
 * Computed blockwise in fp32 (64-row chunks: each key moved to its chunk's end, then through the
 * later chunks' transforms right to left; 32-row chunks at head_dim 128) and rounded once to
 * cache_dtype.
 * k, v, w: [batch][heads][prompt_len][head_dim] in cache_dtype; beta: [batch][heads][prompt_len]
 * float32 (clamped to [0, 2]).  Caches: [batch][heads][capacity][head_dim]; rows >= prompt_len
 * are not touched.  Requires 0 <= prompt_len <= capacity (else PATH_ERR_CAPACITY); prompt_len = 0
 * does nothing.  PaTH-FoX: with log_f ([batch][heads][prompt_len] float32) and a_cache
 * ([batch][heads][capacity] float32) both given, rows 0..prompt_len-1 of a_cache get the inclusive
 * prefix sums of log_f, as path_decode_step_fox expects; both NULL for plain PaTH (one without the
 * other is PATH_ERR_INVALID_ARG).  ws: at least path_decode_prefill_workspace_size(desc, prompt_len) bytes,
 * 256-byte aligned.  Asynchronous on stream.
 */
int path_decode_prefill(const path_decode_desc_t* desc, void* k_cache, void* v_cache, int prompt_len,
                        const void* k, const void* v, const void* w, const float* beta, const float* log_f,
                        float* a_cache, void* ws, size_t ws_bytes, void* stream);

/*
 * One PaTH-FoX decode step (notes §2.8 Eq. (1) with the forget gate of §2.5): the key rewrite
 * and append of path_decode_step, and the logit of cached key j gains
 *   sum_{s=j+1..t} log f_s = a_t - a_j,
 * where a_cache ([batch][heads][capacity] float32) holds the prefix sums a_j = sum_{s<=j} log f_s
 * of the cached rows (rows 0..t-1 on entry; path_decode_prefill with log_f fills them for a
 * prompt).  The step stores a_t = a_{t-1} + log_f_t (a_{-1} = 0) in row t, then
 *   o_t = sum_j softmax_j(scale k_j . q_t + a_t - a_j) v_j   over j = 0..t.
 * log_f_t: [batch][heads] float32 (log of the forget gate, <= 0).  Other arguments, requirements
 * and errors as path_decode_step (same workspace size).
 */
int path_decode_step_fox(const path_decode_desc_t* desc, void* k_cache, void* v_cache, float* a_cache, int t,
                         const void* q_t, const void* k_t, const void* v_t, const void* w_t, const float* beta_t,
                         const float* log_f_t, void* o_t, void* ws, size_t ws_bytes, void* stream);

#define PATH_DECODE_NOALLOC_MAX_HEADS 496
/*
 * path_decode_step without a workspace argument.  The paper has no counterpart: this exists
 * for callers that cannot allocate device memory when they decode — code running inside
 * another runtime's memory pool without access to its allocator, plugins that may only use
 * the buffers handed to them, or serving loops that forbid allocation after start-up.
 *
 * Same arguments, semantics and results as path_decode_step, minus ws/ws_bytes.  The per-split
 * partial softmax states live in a fixed 16 MiB array inside the library, present on every
 * GPU that loads it until the process exits.  Limit: batch * heads <= PATH_DECODE_NOALLOC_MAX_HEADS,
 * otherwise PATH_ERR_WORKSPACE is returned and nothing runs.  The call itself allocates
 * nothing (no cudaMalloc, no library allocator).
 *  - The first call made with a given device current looks up the array's device address
 *    (cudaGetSymbolAddress) and caches it; make that first call before any stream capture.
 *    The cached address belongs to that device's current context: after cudaDeviceReset (or
 *    anything else that destroys the primary context) it is stale, and this entry point must
 *    not be called again in that process.
 *  - All calls on a device share the one array: calls that may overlap on the GPU (different
 *    streams without ordering between them) race and give wrong results.  Calls ordered on one
 *    stream are safe.  Nothing in the array needs to start at zero: each call overwrites the
 *    parts it reads.
 */
int path_decode_step_noalloc(const path_decode_desc_t* desc, void* k_cache, void* v_cache, int t,
                             const void* q_t, const void* k_t, const void* v_t, const void* w_t,
                             const float* beta_t, void* o_t, void* stream);

/*
 * Device-side status of the passes that ran on a workspace.  (The pages have no failure
 * machinery; this is the library's own.)  Every wait of the tensor-core kernels on their internal
 * pipeline barriers is bounded (about 2 s); a wait that gives up writes a nonzero code into an int
 * inside the workspace (the first code wins) and its kernel ends early, so the outputs of that
 * call are incomplete even though the call returned PATH_OK (kernels run after it returns).
 * This call waits for all work queued on `stream` (it synchronises the stream), then reads that
 * word through a 4-byte copy into host memory.
 *   desc, for_backward: the descriptor and the pass the workspace was sized for (they fix where the
 *     word lives); ws, ws_bytes: that workspace.
 * Returns PATH_OK (no wait gave up), PATH_ERR_INTERNAL (one did; *code, when code is not NULL,
 * receives the first recorded code), PATH_ERR_CUDA (the synchronisation or the copy failed, e.g.
 * after a kernel fault), or an argument error as the passes would return it.  Passes that run the
 * fp32 CUDA-core kernels have no such waits: the call returns PATH_OK for them without touching
 * the device.
 * The word is cleared by the forward's PREPARE phase and by the backward's PREPARE phase (except
 * with PATH_BWD_REUSE_FWD or PATH_BWD_Z_FROM_FWD, where it keeps the forward's code), so it covers
 * every tensor-core kernel since the last clearing.
 * Test hook: with the environment variable PATH_ATTN_DEBUG_STALL_NS set to n > 0 at the time of
 * a call, the forward's PREPARE phase on the tensor-core path (and, with code 99 as well, every tensor-core
 * kernel of linear attention; their statuses are below) makes every CTA wait on a barrier
 * that nothing arrives at, give up after n ns (at most 1 s), record code 99 and end without
 * writing anything; the workspace status then reads PATH_ERR_INTERNAL with code 99.  The context
 * stays usable: a later call without the variable runs normally.
 */
int path_attn_workspace_status(const path_attn_desc_t* desc, int for_backward, const void* ws, size_t ws_bytes,
                               int* code, void* stream);

/* The same for the workspace of path_decode_prefill (desc and prompt_len as given to it): the
 * tcgen05 preparation of bf16 caches at head dim 64 has bounded waits; the other hand-off paths
 * have none (PATH_OK).  Synchronises `stream`. */
int path_decode_prefill_status(const path_decode_desc_t* desc, int prompt_len, const void* ws, size_t ws_bytes,
                               int* code, void* stream);

/*
 * Context parallelism (sequence sharding) of the forward pass.  The reading notes §2.8, last
 * paragraph (the paper's Sec. 3.5), sketch it: pass the transported keys and values and the block
 * transforms between devices and accumulate right to left.  The sequence of L tokens is cut into
 * consecutive shards, one per device, each a multiple of 128 tokens.  For a query i of shard r and
 * a key j of an earlier shard r':
 *   logit(i, j) = scale * k~_j^T (M_{r'+1} ... M_{r-1}) z^_i + a_i + b_j
 * with k~_j = H_{e(r')} ... H_{j+1} k_j (the key moved to the end of its shard), z^_i =
 * H_{s(r)} ... H_i q_i (the query moved to the start of its shard), M_s = H_{s(s)} ... H_{e(s)}
 * (the product over shard s) and, with a forget gate, a_i = sum_{t=s(r)..i} log f_t and
 * b_j = sum_{t=j+1..e(r')} log f_t plus the totals of the shards in between.  Each device then:
 *   1. runs path_attn_fwd_phases(PATH_FWD_PREPARE) on its shard (fwd_ws) and
 *      path_cp_shard_prepare (its keys moved to its end, its queries moved to its start, M^T, and
 *      the forget-gate terms);
 *   2. for every earlier shard, receives that shard's key block (already moved to the end of the
 *      previous shard), its values and key biases, merges them into its queries' softmax state
 *      with path_cp_attend_block, moves the block through its own shard with path_cp_pass_block
 *      and sends it on to the next device;
 *   3. runs path_attn_fwd_phases(PATH_FWD_SCAN): o and lse over the whole prefix.
 * The order in which blocks are merged does not change the result (up to rounding).  Scope: bf16
 * at head dim 64 (the tensor-core path), seqlen and block_len multiples of 128, forward only (the
 * backward is not sharded).  desc is always the local shard's descriptor (seqlen = its length).
 */

/* Bytes of workspace path_cp_shard_prepare needs; 0 if desc is invalid or outside the scope. */
size_t path_cp_prepare_workspace_size(const path_attn_desc_t* desc);

/*
 * Per-shard transports.  Inputs q, k, w ([batch][heads][seqlen][64] bf16), beta (fp32), log_f
 * (fp32 or NULL).  Outputs (caller-owned device memory):
 *   k_end   [batch][heads][seqlen][64] fp32: row j = k~_j, the key moved to the shard's end;
 *   q_start [batch][heads][seqlen][64] bf16: row i = z^_i, the query moved to the shard's start;
 *   t_shard [batch][heads][64][64] fp32: M^T, the transpose of the shard's product (row-major);
 *   with log_f (all three or none): a_q [batch][heads][seqlen] = inclusive prefix sums of log f,
 *   b_k = total - a_q, f_tot [batch][heads] = the total.
 * Computed from the UT preparation (split-precision fp32 chunk transforms, as the prefill hand-off)
 * by two fp32 walks over the chunks.  ws: path_cp_prepare_workspace_size bytes, 256-byte aligned,
 * contents unspecified on exit (a bounded wait of its preparation that gives up is recorded there
 * but not reported by a status call).
 * Errors: PATH_ERR_UNSUPPORTED outside the scope above; argument errors as elsewhere.
 */
int path_cp_shard_prepare(const path_attn_desc_t* desc, const void* q, const void* k, const void* w,
                          const float* beta, const float* log_f, float* k_end, void* q_start, float* t_shard,
                          float* a_q, float* b_k, float* f_tot, void* ws, size_t ws_bytes, void* stream);

/* Bytes of block scratch path_cp_attend_block needs for blocks of block_len keys; 0 if invalid. */
size_t path_cp_block_workspace_size(const path_attn_desc_t* desc, int block_len);

/*
 * Merges one earlier shard's key block into the softmax state that the forward's PREPARE phase left
 * in fwd_ws (path_attn_workspace_size(desc, 0 or 1) bytes, the same workspace the later SCAN phase
 * uses): for every local query i (row of q_start) and every block key j,
 *   s_ij = scale * k_block_j . q_start_i (+ a_q_i + b_k_j),
 * added to the query's running maximum, sum and weighted values with v_block_j.  k_block
 * [batch][heads][block_len][64] fp32 (rounded to bf16 for the tensor-core product), v_block the
 * same shape in bf16, a_q [..][seqlen] and b_k [..][block_len] fp32 or both NULL.  blk_ws:
 * path_cp_block_workspace_size bytes, 256-byte aligned.  Runs the forward scan kernel in its block
 * mode (tcgen05); its bounded waits report through path_attn_workspace_status on fwd_ws.
 */
int path_cp_attend_block(const path_attn_desc_t* desc, int block_len, const void* q_start, const float* k_block,
                         const void* v_block, const float* a_q, const float* b_k, void* fwd_ws, size_t fwd_ws_bytes,
                         void* blk_ws, size_t blk_ws_bytes, void* stream);

/*
 * Moves a key block through the local shard, in place: rows k_block <- k_block M (k_block
 * [batch][heads][block_len][64] fp32, t_shard = M^T from path_cp_shard_prepare), and with a forget
 * gate b_k += f_tot (b_k [batch][heads][block_len], f_tot [batch][heads]; both or neither).
 */
int path_cp_pass_block(const path_attn_desc_t* desc, int block_len, float* k_block, float* b_k,
                       const float* t_shard, const float* f_tot, void* stream);

/*
 * Paged serving
 * -------------
 * A cache of many sequences of different lengths, in pages: keys in one pool, values in another, and
 * for every sequence slot one table of page numbers into each.  Row j of slot b lies in page
 * k_table[b][j / page_size] (v_table for its value) at row j % page_size.  As in the dense decode
 * cache, keys are held transported to the newest position, so every step rewrites every key of its
 * sequence: a key page belongs to exactly one sequence.  Values (and the forget gate's running sums,
 * which lie beside the values) never change once written: a value page may be shared.
 *
 * All pointers are device memory of the caller; the lists and tables are read on the device, so that
 * a captured step replays with new contents.  A slot with seq_len < 0 is empty.
 */
typedef struct {
  int slots;        /* sequence slots: rows of the tables, 1..65535 */
  int heads;        /* key/value heads */
  int head_dim;     /* 64 or 128 */
  int page_size;    /* rows of a page: 16, 32, 64, 128 or 256 */
  int table_width;  /* columns of the tables: a slot holds at most table_width * page_size tokens */
  int k_pages;      /* pages of the key pool */
  int v_pages;      /* pages of the value pool */
  int cache_dtype;  /* path_dtype_t of the pools and of q, k, v, w, o */
  void* k_pool;     /* [k_pages][heads][page_size][head_dim] */
  void* v_pool;     /* [v_pages][heads][page_size][head_dim] */
  float* a_pool;    /* [v_pages][heads][page_size]: running sums of log f (PaTH-FoX), or NULL */
  int* k_table;     /* [slots][table_width]; -1: no page */
  int* v_table;     /* [slots][table_width] */
  int* seq_len;     /* [slots]: tokens in the cache; < 0: empty slot */
  int* k_ref;       /* [k_pages]: 1 in use, 0 free */
  int* v_ref;       /* [v_pages]: sequences that hold the page, 0 free */
  int* status;      /* one int: the first PATH_PAGED_* code since it was last cleared (start it at 0) */
  int* extended;    /* [slots] or NULL: tokens that the last path_paged_extend of a slot gave it and no
                       path_paged_advance has counted yet; -1: it left the slot out (start it at 0, and set
                       it to 0 with a seq_len of your own).  NULL: advance cannot tell and counts what its
                       q_start says, as far as there are pages */
  float* a_rest;    /* as a_pool, or NULL: what rounding the running sums to fp32 left of them (0 where the
                       caller fills a_pool itself).  NULL: every call rounds the sums it appends by up to
                       2^-24 of their size, which far into a sequence is more than a token adds */
} path_paged_cache_t;

/* Codes of the status word: what a call found on the device.  None of them makes a kernel leave its
 * buffers; see each call for what it then leaves undone. */
enum {
  PATH_PAGED_BAD_PAGE = 1,    /* a needed table entry is not a page of the pool */
  PATH_PAGED_CAPACITY = 2,    /* a sequence would outgrow table_width * page_size */
  PATH_PAGED_BAD_SLOT = 3,    /* slot out of range, listed twice, empty where it must not be, or in use */
  PATH_PAGED_NO_PAGES = 4,    /* not enough free pages */
  PATH_PAGED_BAD_START = 5,   /* q_start falls, leaves [0, total_tokens] or exceeds max_new; advance: it
                                 is not what extend was given */
  PATH_PAGED_BAD_TOKEN = 6,   /* verify: a drafted token is not in the vocabulary */
  PATH_PAGED_WAIT = 64        /* and above: a bounded wait of a tensor-core kernel gave up */
};

typedef struct {
  int heads_q;       /* query heads, a multiple of cache.heads (at most 16 times): head hq reads key head
                        hq / (heads_q / heads) */
  int total_tokens;  /* new tokens of the call */
  int max_new;       /* at least the most new tokens of one slot.  0 says that there are none: nothing is
                        launched and q_start is not looked at */
  float scale;       /* multiplies the logit; the forget bias is added unscaled */
  int window;        /* 0: every earlier token is seen; W > 0: the token at position p sees j > p - W ... */
  int sinks;         /* ... and the first `sinks` tokens of its sequence */
  int max_multi;     /* at most so many slots have several new tokens (0: any number).  Others beyond them may
                        be left out with PATH_PAGED_BAD_START.  What the workspace of a call with max_new > 1
                        is for: unstated, it holds half as many slots as there are new tokens, in rounds of
                        what about 4 GiB hold */
} path_paged_desc_t;

/* Bytes of workspace path_paged_extend needs; 0 if cache or desc is invalid.  Host only. */
size_t path_paged_workspace_size(const path_paged_cache_t* cache, const path_paged_desc_t* desc);

/*
 * Attention of new tokens over the paged cache: a prompt chunk, a few draft tokens or one token per
 * sequence, in any mixture.  Tokens are packed: q, o [total_tokens][heads_q][head_dim], k, v, w
 * [total_tokens][heads][head_dim] in cache_dtype, beta (clamped to [0, 2]) and log_f (NULL exactly when
 * a_pool is) [total_tokens][heads] float32.  Slot b's new tokens are q_start[b] .. q_start[b + 1] - 1 (int32
 * [slots + 1]); they take positions seq_len[b] and up.  q_start NULL: one token per slot, token b for
 * slot b (total_tokens = slots), empty slots skipped (their rows of o are not written).
 * With H_t = I - beta_t w_t w_t^T, for every token at position p of a slot,
 *   o_p = sum_j softmax_j(scale k_j^T H_{j+1} ... H_p q_p  (+ a_p - a_j)) v_j   over the j <= p it sees;
 * afterwards the new rows are appended (keys transported to the last new token) and every cached key
 * that a later token sees is k_j <- H_last ... H_first k_j, rounded once per call (bf16: once for every
 * 4096 new tokens of the slot, which are taken in that many passes).  Keys that the window hides from
 * every later token are left as they are (new ones: as appended, or as the pass stored them); their
 * table entries may be -1.
 * seq_len is read, not changed (path_paged_advance does that).  The pages must be there
 * (path_pages_reserve).  A slot whose row of q_start or length is bad, or that lacks a page for one of
 * its new tokens, is left out whole: nothing of it is read into o or written, and advance passes it
 * over.  Cached rows whose page is missing are treated as hidden and are not written.  Status gets the
 * code.  Ranges of q_start that overlap mix those slots' results; with more tokens in them than
 * total_tokens, slots with several tokens are left out and status gets PATH_PAGED_BAD_START.
 * The cached keys pass all tokens of the call, and nothing takes that back: draft tokens of which
 * some may be rejected are given to a fork of their sequence (path_pages_fork), and those accepted then
 * to the sequence itself (or, where all are, the fork stays in its place).
 * o must not overlap the inputs or the pools.
 * Pool rows behind seq_len and pages that no table names may hold anything.  An infinity or NaN in a
 * slot's own tokens or cached rows may reach any output of that slot, never another slot's.
 * ws: at least path_paged_workspace_size(cache, desc) bytes, 256-byte aligned.  Two calls that may
 * run at the same time need two workspaces (and must not share a slot).
 */
int path_paged_extend(const path_paged_cache_t* cache, const path_paged_desc_t* desc, const int* q_start,
                      const void* q, const void* k, const void* v, const void* w, const float* beta,
                      const float* log_f, void* o, void* ws, size_t ws_bytes, void* stream);

/*
 * seq_len[b] += q_start[b + 1] - q_start[b] for the slots in use (q_start NULL: += 1), with the q_start
 * of the extend before it.  A slot that extend left out is passed over; one that it gave another number of
 * tokens gets PATH_PAGED_BAD_START and keeps its length.  Without an extend before it (rows that the
 * caller wrote itself) the rows' pages have to be there (PATH_PAGED_BAD_PAGE).
 */
int path_paged_advance(const path_paged_cache_t* cache, const int* q_start, void* stream);

/*
 * Reads the status word (synchronises the stream) and clears it.  PATH_OK with *code 0; or *code is
 * the first code recorded: PATH_ERR_INVALID_ARG for BAD_PAGE, BAD_SLOT and BAD_START, PATH_ERR_CAPACITY
 * for CAPACITY and NO_PAGES, PATH_ERR_INTERNAL from PATH_PAGED_WAIT on.
 */
int path_paged_status(const path_paged_cache_t* cache, int* code, void* stream);

/* Bytes of workspace the path_pages_* calls need; 0 if cache is invalid.  Host only. */
size_t path_pages_workspace_size(const path_paged_cache_t* cache);

/*
 * Page management.  Lists are int32 device arrays.  Pages are given out lowest free number first, in
 * the order of the list (of the slots) and then of the columns.  A call that records a code changes
 * nothing (path_paged_advance: nothing of that slot).  ws: at least path_pages_workspace_size(cache)
 * bytes, 256-byte aligned.
 *
 * reserve: pages for n_new[b] more tokens ([slots], NULL: 1 for every slot in use) behind seq_len[b]; an
 *   empty slot with n_new[b] > 0 is opened with length 0.
 * fork: children[i] (an empty slot, listed once) becomes a copy of parents[i] (a slot in use; it may have
 *   several children).  Its keys are copied to new pages, because the next step rewrites them; full
 *   value pages are shared, a partly filled last one is copied with its running sums.  Reserved pages
 *   behind the parent's last row are not taken over.
 * free: the slots become empty and their pages return (a shared value page with its last holder).
 * trim: returns the pages of every slot in use that hold only rows which a window of `window` tokens
 *   and `sinks` first tokens hides from every later token; their table entries become -1.  The page
 *   of the last row stays.  Positions go on: the columns are not given back, and a slot ends at table_width
 *   * page_size tokens whatever the window.
 * compact: moves the pages in use to the front of each pool: with n pages in use, those numbered n and
 *   above go, in rising order, to the free numbers below n.  Tables and counts follow.
 */
int path_pages_reserve(const path_paged_cache_t* cache, const int* n_new, void* ws, size_t ws_bytes, void* stream);
int path_pages_fork(const path_paged_cache_t* cache, const int* parents, const int* children, int count, void* ws,
                    size_t ws_bytes, void* stream);
int path_pages_free(const path_paged_cache_t* cache, const int* slots, int count, void* ws, size_t ws_bytes,
                    void* stream);
int path_pages_trim(const path_paged_cache_t* cache, int window, int sinks, void* ws, size_t ws_bytes, void* stream);
int path_pages_compact(const path_paged_cache_t* cache, void* ws, size_t ws_bytes, void* stream);

/*
 * A step's plan: path_pages_reserve(n_new), and where the new tokens go, for tokens packed in slot order.
 * n_new [slots], negative values count as 0, or NULL: 1 for every slot in use.  All outputs are written whole:
 *   q_start [slots + 1]: running sums of n_new;
 *   slot, position [tokens]: each packed token's slot and position in its sequence (seq_len + its number);
 *   k_row, v_row [tokens]: its row in each pool, page * page_size + place in the page (head h of it is row
 *     place of [page][h]);
 *   source [tokens] with from_start [slots + 1], or both NULL: from_start[slot] + its number, its row in an
 *     earlier packing that began with the same tokens of each slot (draft tokens, say, of which n_new were kept).
 * What stands behind the last token is -1.  tokens: what the arrays hold.  With more new tokens than that
 * (PATH_PAGED_BAD_START), and where reserve records a code, no page is given out, q_start is 0 and the maps are -1.
 * ws as for path_pages_reserve.
 */
int path_pages_plan(const path_paged_cache_t* cache, const int* n_new, const int* from_start, int tokens, int* q_start,
                    int* slot, int* position, int* k_row, int* v_row, int* source, void* ws, size_t ws_bytes,
                    void* stream);

/*
 * Verification of drafted tokens: which of them a target model keeps, and the token after them, so that what is
 * kept is distributed as if the target had drawn it.  A slot's packed tokens q_start[b] .. q_start[b + 1] - 1 (as
 * given to path_paged_extend) are one that is known, then its drafts; row i of target holds the target's
 * probabilities of the token after token i, row i of draft those that token i was drawn from (of a slot's first
 * token: not read).  draft NULL: the drafts are certain, their probability is 1.
 *   Draft i is kept if all before it are and uniform[i] * draft[i][x] < target[i - 1][x], x = tokens[i].
 *   keep[b]: tokens kept, the known one among them (1 .. count; 0: the slot has none).
 *   next[b]: drawn with uniform[q_start[b]] from max(0, target - draft) of the first draft not kept (where that
 *     is 0 throughout: from target), or from target's last row where all are kept: the lowest x at which the
 *     running sum exceeds uniform * the row's sum.  -1: the slot has no token, or the row no positive entry.
 * Products, differences and sums are exact to 2^-40 and better.  Probabilities need not add up to 1; NaN and negative ones
 * count as 0.  A draft outside [0, vocab) is not kept (PATH_PAGED_BAD_TOKEN; none is taken out of its row).  A slot
 * whose row of q_start is bad gets 0 and -1 (PATH_PAGED_BAD_START).
 * The rows are probabilities: of logits, a softmax comes before this call and moves every row twice, where this call
 * reads the one or two rows of a slot that decide.
 */
typedef struct {
  int slots;          /* 1..65535 */
  int total_tokens;   /* rows of target and draft, entries of tokens and uniform */
  int max_new;        /* at least the most tokens of one slot */
  int vocab;          /* entries of a row, 1..2^20 */
  int dtype;          /* path_dtype_t of target and draft */
  long long target_stride, draft_stride; /* entries from a row to the next, at least vocab */
} path_verify_desc_t;
int path_draft_verify(const path_verify_desc_t* desc, const int* q_start, const int* tokens, const float* uniform,
                      const void* target, const void* draft, int* keep, int* next, int* status, void* stream);

/*
 * Linear attention
 * ----------------
 * With a decay g = exp(log_decay[h]) per key head and a state S (head_dim x head_dim, float32):
 *   S_t = g S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t.
 * log_decay [heads] float32, natural log, kept in [-10000, 0]; NaN makes its head's outputs NaN.  An infinity or NaN in
 * a sequence may reach any output of that sequence and head, of earlier tokens too.
 * Results are the same from call to call.  How a sequence is cut and, in bf16, how often a weight is rounded goes by the
 * sizes of the whole call: beside others a sequence may get other last bits than alone, within the same bounds.
 */
typedef struct {
  int batch, heads_q;  /* heads_q: a multiple of heads (at most 16 times); head hq reads key head hq / (heads_q / heads) */
  int heads, seqlen;
  int head_dim;        /* 64 or 128 */
  int dtype;           /* path_dtype_t of q, k, v, o and the gradients */
  float scale;
} path_linear_desc_t;

/* Bytes of workspace of path_linear_fwd (for_backward 0) or path_linear_bwd (1); 0 if desc is invalid.  Host only. */
size_t path_linear_workspace_size(const path_linear_desc_t* desc, int for_backward);
/* o from a zero state.  q, o [batch][heads_q][seqlen][head_dim], k, v [batch][heads][seqlen][head_dim]. */
int path_linear_fwd(const path_linear_desc_t* desc, const void* q, const void* k, const void* v, const float* log_decay,
                    void* o, void* ws, size_t ws_bytes, void* stream);
/* Gradients of q, k and v (a key head's summed over its query heads); log_decay is a constant of the model.
 * Those of dq, dk and dv that are NULL are not computed (one at least is not). */
int path_linear_bwd(const path_linear_desc_t* desc, const void* q, const void* k, const void* v, const float* log_decay,
                    const void* dO, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes, void* stream);
/* As path_attn_workspace_status, of the call that ran on ws last: with a code (PATH_PAGED_WAIT and above), what it wrote is
 * incomplete. */
int path_linear_workspace_status(const path_linear_desc_t* desc, const void* ws, size_t ws_bytes, int* code, void* stream);

/* States of many sequences, for serving: the slots' states in place of their tokens. */
typedef struct {
  int slots, heads;    /* slots 1..65535 */
  int head_dim;        /* 64 or 128 */
  int dtype;           /* path_dtype_t of q, k, v, o */
  float* state;        /* [slots][heads][head_dim (of k)][head_dim (of v)] */
  int* status;         /* one int, as in path_paged_cache_t */
} path_linear_cache_t;
typedef struct {
  int heads_q, total_tokens, max_new;  /* as in path_paged_desc_t */
  float scale;
  int update;          /* 0: the states stay (draft tokens of which some may be rejected) */
} path_linear_step_t;

/* Bytes of workspace path_linear_extend needs; 0 if cache or step is invalid.  Host only. */
size_t path_linear_extend_workspace_size(const path_linear_cache_t* cache, const path_linear_step_t* step);
/*
 * New tokens of many sequences, packed as for path_paged_extend: q, o [total_tokens][heads_q][head_dim], k, v
 * [total_tokens][heads][head_dim], slot b's being q_start[b] .. q_start[b + 1] - 1 (NULL: token b is slot b's).
 * A slot whose row of q_start is bad, or begins before an earlier good row's tokens end, is left out whole
 * (PATH_PAGED_BAD_START).  o must not overlap the inputs or the states.  ws: for one call at a time; not used, and may
 * be NULL, with a max_new of at most 16.  An infinity or NaN in a slot's tokens or state may reach any output of that
 * slot, never another's.
 */
int path_linear_extend(const path_linear_cache_t* cache, const path_linear_step_t* step, const int* q_start, const void* q,
                       const void* k, const void* v, const float* log_decay, void* o, void* ws, size_t ws_bytes,
                       void* stream);
/* children[i] takes the state of parents[i] (NULL: zeros, a new sequence).  An entry that names no slot, or a child
 * that is listed twice or is a parent too, is left out (PATH_PAGED_BAD_SLOT). */
int path_linear_fork(const path_linear_cache_t* cache, const int* parents, const int* children, int count, void* stream);
/* As path_paged_status.  After a code of PATH_PAGED_WAIT and above the outputs and the states of that call's slots are not
 * to be used. */
int path_linear_status(const path_linear_cache_t* cache, int* code, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PATH_ATTN_H */
