/*
 * attn.h -- C ABI of libattn.so: fused causal scaled-dot-product attention
 * (forward, backward, LSE merge), the norm and rotation of its queries and
 * keys, and attention over a paged 4-bit cache (shared prefixes, eviction), for
 * NVIDIA GB300 (sm_103a).
 *
 * Sources for the operations (web pages on Blackwell attention backends):
 *  - TransformerEngine PR #3527, "cuDNN FROST attention backend for head_dim in
 *    (256, 512], with context parallelism": forward with a natural-log FP32
 *    log-sum-exp; graphs built from each tensor's actual strides; output
 *    buffers owned by the caller; unsupported configurations refused rather
 *    than approximated; k/v stride agreement and GQA divisibility checks;
 *    sliding window (left, right) with -1 unbounded and a causal mask pinning
 *    the right bound to the diagonal; top-left / bottom-right causal alignment;
 *    the stream bound per call; a context-parallel ring merging partial
 *    results through LSE differences.
 *  - TransformerEngine PR #3699, "cuDNN FROST D128/D256 backward dispatch":
 *    the backward helper chain (the D = rowsum(dO * O) preprocess, gradient
 *    reductions over GQA groups), per-execution device checks of cu_seqlens,
 *    pointers / stream / workspace bound per call, exactly zero dQ on rows
 *    that see no key.
 *  - TransformerEngine PR #3149, "FA4 for context parallelism": packed THD
 *    tensors addressed through cu_seqlens.
 *
 * Conventions for every entry point:
 *  - All tensor pointers are DEVICE pointers owned by the caller.  The library
 *    allocates no memory and keeps no state between calls (except a
 *    thread-local error string and a cached driver entry point).
 *  - Work is enqueued on `stream`; calls return once it is enqueued.
 *  - A problem the host can see (bad shape, stride, alignment, dtype, head
 *    dim, workspace) is returned at once and nothing is launched.
 *  - A problem only the device can see (inconsistent cu_seqlens, a wait that
 *    exceeded its time limit) is written to the status word at the start of
 *    the workspace; the kernels then stop early and leave the outputs
 *    undefined.  attn_query_status() reads it.  No kernel ever traps.
 *  - Element strides are given as {batch, token, head}; the head-dim axis is
 *    contiguous.  Q/K/V/O/dO/dQ/dK/dV may each have their own strides.
 *  - Dense layout (cu_seqlens NULL): tensors are [batch][seqlen][heads][d].
 *    Varlen THD layout (cu_seqlens set): tensors are [total][heads][d] and
 *    sequence b owns rows [cu_seqlens[b], cu_seqlens[b+1]); the batch stride
 *    is ignored.
 *  - LSE is FP32 natural log.  Default layout [batch][heads_q][seqlen_q]
 *    (dense) or [heads_q][total_q] (THD); stride_lse overrides it.
 *  - A query row that sees no key gets O = 0, LSE = -inf and dQ = 0.
 */
#ifndef ATTN_H_
#define ATTN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* attn_stream_t; /* a cudaStream_t; NULL = legacy default stream */

typedef enum {
  ATTN_OK = 0,
  ATTN_ERR_INVALID_ARG = 1,  /* null pointer, negative size, inconsistent shape */
  ATTN_ERR_UNSUPPORTED = 2,  /* valid request this library refuses (head dim, dtype mix) */
  ATTN_ERR_ALIGNMENT = 3,    /* pointer or stride not 16-byte aligned as required */
  ATTN_ERR_WORKSPACE = 4,    /* workspace missing or smaller than *_workspace_size() */
  ATTN_ERR_BAD_METADATA = 5, /* device check: cu_seqlens inconsistent, or an index out of
                                range (status word) */
  ATTN_ERR_TIMEOUT = 6,      /* device wait exceeded its time limit (status word) */
  ATTN_ERR_CUDA = 7          /* a CUDA runtime call failed; see attn_last_error() */
} attn_status_t;

typedef enum { ATTN_BF16 = 0, ATTN_FP16 = 1, ATTN_FP32 = 2 } attn_dtype_t;

typedef struct {
  attn_dtype_t dtype;      /* Q, K, V, dO: ATTN_BF16 or ATTN_FP16 */
  attn_dtype_t o_dtype;    /* O: == dtype, or ATTN_FP32 (partials for attn_lse_merge) */
  attn_dtype_t grad_dtype; /* dQ, dK, dV: == dtype, or ATTN_FP32 */
  int batch;               /* dense: batch size; THD: number of sequences */
  int seqlen_q, seqlen_k;  /* dense: sequence lengths; THD: maximum lengths */
  const int32_t* cu_seqlens_q; /* device [batch+1] prefix sums, or NULL for dense */
  const int32_t* cu_seqlens_k; /* device [batch+1]; must be set iff cu_seqlens_q is */
  int total_q, total_k;    /* THD: rows of the packed tensors (== cu_seqlens[batch]) */
  int heads_q, heads_kv;   /* heads_q % heads_kv == 0; query head h uses kv head h/(hq/hkv) */
  int d_qk, d_v;           /* (64,64) (128,128) (192,128) (256,256) (512,512) */
  int64_t stride_q[3], stride_k[3], stride_v[3], stride_o[3]; /* {batch, token, head} */
  int64_t stride_do[3], stride_dq[3], stride_dk[3], stride_dv[3];
  int64_t stride_lse[2];   /* {batch, head} in elements; {0, 0} = default layout */
  int causal;              /* 1: key j visible only if j <= i + off */
  int bottom_right;        /* off = seqlen_k - seqlen_q (per sequence) if 1, else 0 */
  int window_left;         /* visible only if j >= i + off - window_left; -1 unbounded */
  int window_right;        /* visible only if j <= i + off + window_right; -1 unbounded */
  float softmax_scale;     /* > 0, typically 1/sqrt(d_qk) */
  int accumulate;          /* attn_bwd with grad_dtype FP32 only: 1 adds the gradients
                              into dq/dk/dv instead of overwriting them (used to sum
                              the partial gradients of a context-parallel ring) */
  const int32_t* seqused_q; /* THD only, device [batch] or NULL: padded layout (PR #3149:
                               physical padded offsets plus visible lengths).  Sequence b
                               then uses rows [cu_seqlens_q[b], cu_seqlens_q[b] +
                               seqused_q[b]); the rows up to cu_seqlens_q[b+1] are a gap
                               that no kernel reads or writes. */
  const int32_t* seqused_k; /* the same for keys/values; set both or neither */
  int bwd_ds;              /* backward at head dims (128,128) and (192,128): 0 = auto
                              (keep dS in the workspace when its blocks take at most
                              64 GiB), 1 = keep dS, -1 = never (recompute the scores
                              for dQ: the smallest workspace).  See attn_bwd_path. */
} attn_params_t;

/* Bytes of workspace attn_fwd / attn_bwd need for `p` (always >= 256: the
 * status word lives at offset 0).  The workspace must be 256-byte aligned.
 * On the ATTN_BWD_PDS path the backward also keeps P and dS of every visible
 * 128-query x 128-key tile (64 KiB each, all query heads) in the workspace,
 * on the ATTN_BWD_DS path dS alone (32 KiB each): the count is exact for
 * dense inputs, and for THD it is a bound that takes every document's keys
 * as max_seqlen_k long (P and dS: about 8.7 GB for batch 1, 16 query heads,
 * 16384 causal tokens; dS: about 34.5 GB for batch 1, 32 query heads, 32768
 * causal tokens). */
size_t attn_fwd_workspace_size(const attn_params_t* p);
size_t attn_bwd_workspace_size(const attn_params_t* p);

/* The backward that attn_bwd runs for `p` (a pure function of `p`):
 *   ATTN_BWD_RECOMPUTE  a query-stationary dQ kernel and a key-stationary
 *                       dK/dV kernel that both compute S and dP;
 *   ATTN_BWD_DS         head dims (128,128) and (192,128) as bwd_ds allows:
 *                       the dK/dV kernel also writes dS (16-bit)
 *                       into the workspace and dQ = scale dS K is a GEMM over
 *                       it, so S and dP are computed once per query-key pair;
 *   ATTN_BWD_PDS        head dim 512, and 256 while its blocks take at most
 *                       16 GiB: P and dS are written to the workspace and the
 *                       five contractions run once each.
 * All three give results within the same bound of the exact gradients, each
 * bitwise reproducible; they differ in rounding order.  Returns -1 for
 * invalid params. */
typedef enum {
  ATTN_BWD_RECOMPUTE = 0,
  ATTN_BWD_DS = 1,
  ATTN_BWD_PDS = 2
} attn_bwd_path_t;
int attn_bwd_path(const attn_params_t* p);

/*
 * Forward (PR #3527): O = softmax(scale * Q K^T + mask) V per (sequence, query
 * head) with an online softmax over 128-key tiles, and LSE = ln sum_j exp(s_ij)
 * over visible keys.  q, k, v: dtype; o: o_dtype; lse: FP32.  The result is
 * bitwise reproducible (no atomics, fixed reduction order).
 * Alignment: every base pointer 16-byte aligned; every token/head/batch stride
 * a multiple of 8 elements (16-bit tensors) or 4 (FP32 O).
 */
attn_status_t attn_fwd(const attn_params_t* p, const void* q, const void* k, const void* v,
                       void* o, float* lse, void* workspace, size_t workspace_bytes,
                       attn_stream_t stream);

/*
 * Backward (PR #3510 head-parallel backward, PR #3699 helper chain): from Q,
 * K, V, O, dO and the forward's LSE computes D = rowsum(dO * O) (FP32, kept in
 * the workspace beside each row's LSE in base 2, the pair the later kernels
 * read), then per visible tile P = exp(scale QK^T - LSE),
 * dP = dO V^T, dS = P (dP - D), dV = P^T dO, dK = scale dS^T Q,
 * dQ = scale dS K; dK/dV are summed over the query heads of a GQA group
 * inside the kernel.  dq/dk/dv are fully overwritten (grad_dtype).  The
 * reduction order is fixed, so the backward is bitwise reproducible.
 * attn_bwd_path tells which kernels run.  On the ATTN_BWD_PDS path (head dim
 * 512, PR #3527: the d512 backward; head dim 256 up to 16 GiB of blocks) P and
 * dS are written once to the workspace (16-bit, as the fused kernels round
 * them too) and the five contractions run in three kernels; on the
 * ATTN_BWD_DS path the dK/dV kernel writes dS and a GEMM forms dQ from it.  A
 * workspace whose block table does not fit sets ATTN_ERR_WORKSPACE in the
 * status word.
 */
attn_status_t attn_bwd(const attn_params_t* p, const void* q, const void* k, const void* v,
                       const void* o, const void* dout, const float* lse, void* dq, void* dk,
                       void* dv, void* workspace, size_t workspace_bytes, attn_stream_t stream);

/*
 * The three stages of attn_bwd, callable one by one with the same arguments
 * (attn_bwd == preprocess, then dq, then dkdv, on one stream; on the
 * ATTN_BWD_DS path preprocess, then dkdv, then dq):
 *   attn_bwd_preprocess: D = rowsum(dO * O) and LSE * log2 e per query row
 *                        into the workspace; resets the status word (PR #3699
 *                        "backward helper chain");
 *   attn_bwd_dq:         dQ (reads D and LSE from the workspace);
 *   attn_bwd_dkdv:       dK and dV, reduced over each GQA group (reads D and
 *                        LSE from the workspace).
 * The dq and dkdv stages require a preprocess earlier on the stream, on the
 * same workspace, for a problem with the same query rows, query heads, dtype,
 * batch/cu_seqlens_q layout and LSE: D and LSE depend only on each query row,
 * so one preprocess serves several calls that differ only in their keys, mask
 * or window (a context-parallel ring does this; its LSE is the merged one).
 * The dq and dkdv stages ignore their `lse` argument.  Where the backward
 * materialises P and dS (head dim 512; head dim 256 up to 16 GiB of blocks)
 * the dq stage also writes them, with their block plan, into the workspace
 * and the dkdv stage reads them: it then requires the dq stage of the same
 * problem earlier on the stream as well.  On the ATTN_BWD_DS path it is the
 * other way round: the dkdv stage writes dS and its block plan, and the dq
 * stage requires the dkdv stage of the same problem earlier on the stream.
 * Arguments a stage does not use may be NULL.
 */
attn_status_t attn_bwd_preprocess(const attn_params_t* p, const void* q, const void* k,
                                  const void* v, const void* o, const void* dout,
                                  const float* lse, void* dq, void* dk, void* dv,
                                  void* workspace, size_t workspace_bytes, attn_stream_t stream);
attn_status_t attn_bwd_dq(const attn_params_t* p, const void* q, const void* k, const void* v,
                          const void* o, const void* dout, const float* lse, void* dq, void* dk,
                          void* dv, void* workspace, size_t workspace_bytes,
                          attn_stream_t stream);
attn_status_t attn_bwd_dkdv(const attn_params_t* p, const void* q, const void* k, const void* v,
                            const void* o, const void* dout, const float* lse, void* dq,
                            void* dk, void* dv, void* workspace, size_t workspace_bytes,
                            attn_stream_t stream);

/*
 * attn_bwd for callers that cannot allocate device memory (this entry point
 * has no counterpart on the attention pages; it is a deployment aid).
 *
 * Some callers are not allowed to call cudaMalloc while they run: cudaMalloc
 * may synchronise the whole device and takes an unbounded time, so serving
 * loops with latency budgets, plugin hosts that plan every byte of device
 * memory up front, and code running inside another runtime's callbacks
 * forbid it -- and such callers often have no allocator of their own from
 * which to hand attn_bwd a workspace.  attn_bwd_noalloc takes the same
 * arguments as attn_bwd minus the workspace and uses instead a scratch area
 * that the library reserves statically: 8 MiB of device memory per GPU that
 * loads the library, held until the process exits.  That covers problems
 * whose attn_bwd_workspace_size() is at most 8 MiB (about one million
 * query rows x query heads); larger ones return ATTN_ERR_WORKSPACE and
 * nothing is launched.  With bwd_ds = 0 it takes the ATTN_BWD_RECOMPUTE
 * path (the ATTN_BWD_DS path's blocks rarely fit).  It calls no allocating
 * routine.
 *
 * The first call on each device looks up the scratch area's device address
 * (with that device current) and caches it; make that first call before any
 * stream capture.  Every call on a device shares the one scratch area and
 * the status word in it, so calls whose work overlaps on the GPU (different
 * streams, or host threads) race with each other: serialise them.  The
 * status word is cleared at the start of each call; as the caller holds no
 * pointer to it, device-detected problems (inconsistent cu_seqlens, a wait
 * past its limit) are not reported to it -- use attn_bwd where that matters.
 * Results are identical to attn_bwd's.
 */
attn_status_t attn_bwd_noalloc(const attn_params_t* p, const void* q, const void* k,
                               const void* v, const void* o, const void* dout, const float* lse,
                               void* dq, void* dk, void* dv, attn_stream_t stream);

/*
 * One forward + backward step from HOST buffers (a deployment aid with no
 * counterpart on the attention pages: the end-to-end path of a caller whose
 * tensors live in host memory).
 *
 * q, k, v, dout (inputs) and o, lse, dq, dk, dv (outputs) are HOST pointers,
 * laid out with the strides, dtypes and LSE layout that `p` gives, exactly as
 * attn_fwd / attn_bwd would take them on the device; for THD inputs
 * p->cu_seqlens_q/k (and seqused_q/k) are HOST arrays here too.  On `stream`,
 * in order: every input is copied into `arena` (one cudaMemcpyAsync per
 * tensor, the span from its base to its last element), attn_fwd and attn_bwd
 * run there, and O, LSE, dQ, dK, dV are copied back.  With p->accumulate the
 * host dq/dk/dv are uploaded first and the gradients are added to them.
 *
 * arena: caller-owned DEVICE memory, 256-byte aligned, at least
 * attn_host_arena_size(p) bytes: the forward's workspace (its first 256 bytes),
 * then the backward's, then the device copies of all nine tensors.  So
 * attn_query_status(arena) reports device-detected problems of the forward and
 * attn_query_status((char*)arena + 256) those of the backward.  The call
 * returns once the work is enqueued.  Host buffers, and for THD the host
 * cu_seqlens / seqused arrays, should be pinned (cudaHostAlloc /
 * cudaHostRegister) for the copies to be asynchronous: a copy from pageable
 * memory holds the calling thread until the stream has drained, which
 * serialises a pipeline of steps on several streams.  The inputs must not change and the
 * outputs must not be read until the stream has passed the call.  Two calls on
 * two streams with two arenas overlap one step's copies with the other's
 * kernels.  A device pointer among the buffers is refused with
 * ATTN_ERR_INVALID_ARG.  Results are identical to attn_fwd + attn_bwd on the
 * device copies.  attn_host_arena_size returns 0 for parameters that
 * attn_fwd / attn_bwd would refuse.
 */
size_t attn_host_arena_size(const attn_params_t* p);
attn_status_t attn_fwd_bwd_host(const attn_params_t* p, const void* q, const void* k,
                                const void* v, const void* dout, void* o, float* lse, void* dq,
                                void* dk, void* dv, void* arena, size_t arena_bytes,
                                attn_stream_t stream);

/*
 * attn_fwd_bwd_host in stages, for callers that pipeline consecutive steps:
 * `stages` is a mask of ATTN_HOST_UPLOAD (the host inputs, metadata and, with
 * accumulate, the host gradients into the arena), ATTN_HOST_COMPUTE (attn_fwd
 * and attn_bwd on the arena's copies) and ATTN_HOST_DOWNLOAD (O, LSE, dQ, dK,
 * dV back to host memory); ATTN_HOST_ALL is attn_fwd_bwd_host.  Each stage
 * enqueues on `stream`, so a caller can upload step s+1 on one stream while
 * step s computes on another and step s-1 downloads on a third, ordering
 * them with its own events; one arena must not be uploaded into while its
 * previous step still computes or downloads.  The same parameters (shape,
 * strides, flags) must be passed to every stage of one step; the buffers a
 * stage does not touch may be NULL.
 */
enum { ATTN_HOST_UPLOAD = 1, ATTN_HOST_COMPUTE = 2, ATTN_HOST_DOWNLOAD = 4, ATTN_HOST_ALL = 7 };
attn_status_t attn_fwd_bwd_host_stages(const attn_params_t* p, const void* q, const void* k,
                                       const void* v, const void* dout, void* o, float* lse,
                                       void* dq, void* dk, void* dv, void* arena,
                                       size_t arena_bytes, unsigned stages, attn_stream_t stream);

/*
 * LSE-weighted merge of partial attention results over disjoint key sets
 * (PR #3527: the context-parallel ring correction exponentiates LSE
 * differences):  LSE = ln sum_p exp(LSE_p),  O = sum_p exp(LSE_p - LSE) O_p,
 * with the maximum subtracted first; a part whose LSE is -inf has weight 0 and
 * a row with no finite part gets O = 0, LSE = -inf.
 *   o_parts[p]:   device FP32 [part_rows[p]][heads][d_v], contiguous
 *   lse_parts[p]: device FP32 [heads][part_rows[p]], contiguous
 *   part part p covers output rows [part_row0[p], part_row0[p] + part_rows[p])
 *   o_out: [rows][heads][d_v] of o_dtype (BF16, FP16 or FP32), contiguous
 *   lse_out: [heads][rows] FP32.
 * The pointer and range arrays are HOST arrays of n_parts entries
 * (1 <= n_parts <= 64); d_v % 4 == 0.
 */
attn_status_t attn_lse_merge(int n_parts, const float* const* o_parts,
                             const float* const* lse_parts, const int64_t* part_row0,
                             const int64_t* part_rows, int64_t rows, int heads, int d_v,
                             void* o_out, attn_dtype_t o_dtype, float* lse_out,
                             attn_stream_t stream);

/*
 * Local data movement of the all-to-all context-parallel path (PR #3527: after
 * the all-to-all each rank holds the full sequence for a subset of heads), for
 * the cp ranks of a dual-chunk-swap layout held in device memory:
 *   sequence side: rank r holds global chunks r and 2cp-1-r (chunk =
 *     seqlen / (2 cp)) as its local tokens [0, chunk) and [chunk, 2 chunk),
 *     all `heads` heads;
 *   head side:     rank r holds heads [r*heads/cp, (r+1)*heads/cp) of every
 *     token, in sequence order.
 * to_heads = 1 copies sequence side -> head side (src is the sequence side),
 * 0 the reverse.  Each side is described by element strides {rank, token,
 * head}; the d elements of one (token, head) are contiguous and elem_bytes
 * wide (2 for BF16/FP16 tensors, 4 for FP32 such as LSE, which is d = 1 with
 * head-major strides).  A bit-preserving copy; src and dst must not overlap.
 * Requirements: cp >= 1, seqlen a positive multiple of 2 cp, heads % cp == 0,
 * elem_bytes 2 or 4, pointers aligned to elem_bytes.
 */
attn_status_t attn_cp_relayout(int to_heads, int cp, int64_t seqlen, int heads, int d,
                               int elem_bytes, const void* src, const int64_t src_strides[3],
                               void* dst, const int64_t dst_strides[3], attn_stream_t stream);

/* ------------------------------------------------------------------------
 * Around the attention calls: queries and keys before them, and a cache of
 * keys and values held in 4 bits for attention of a few new tokens at a time.
 *
 * These entry points take an optional device word `status` (int32, or NULL).
 * It is sticky: a call never clears it, and sets it to a non-zero value when
 * the device meets a length, position, slot or page that is out of range;
 * attn_query_status(status) reports that as ATTN_ERR_BAD_METADATA.  Zero it
 * once and look at it when convenient.  Nothing out of range is read or
 * written either way.
 * ------------------------------------------------------------------------ */

/*
 * Norm of each query and key head and rotation by its position, in one pass.
 * For every row x (token, head; head_dim elements), in FP32:
 *     y = x / sqrt(mean(x^2) + eps) * w        (norm = 0: y = x, w = NULL)
 *     z = y turned by the angles of the token's position on its first
 *         rotary_dim elements: pairs (i, i + rotary_dim/2), or (2i, 2i+1) with
 *         interleaved = 1:  (a, b) -> (a cos - b sin, b cos + a sin)
 * rounded once to dtype.  At eps = 0 a row whose mean square is 0 in FP32 (below
 * 2^-150) gives zeros, in the gradient too.  A NaN in a row makes all of it NaN; a
 * mean square beyond FP32's range leaves zeros, and NaN for what was infinite.
 * cos/sin: FP32 [max_pos][rotary_dim/2], contiguous,
 * 16-byte aligned (make them in FP64: angles of far positions need it).
 * positions: int32 [batch][seqlen], contiguous, or NULL for 0, 1, .. in each
 * sequence (packed THD tensors: batch 1, seqlen = total).  A negative position
 * marks padding: its rows are neither read nor written.  A position >= max_pos
 * gives NaN rows and sets the status word (with max_pos = 0 all do, and cos and sin
 * may be NULL).
 * w_q / w_k: [head_dim] of w_dtype (FP32 or dtype), or NULL for ones.
 * q, k (and their strides) as in attn_fwd; heads_k may be 0 (queries alone),
 * then the k arguments are ignored.  Views of one projection are fine.
 * z may be written over x (q_out == q with the same strides); any other
 * overlap of an output is refused.
 * head_dim 64, 128, 192, 256 or 512; rotary_dim a multiple of 16 up to head_dim, or 0.
 */
typedef struct {
  attn_dtype_t dtype;    /* q, k, q_out, k_out and gradients: BF16 or FP16 */
  attn_dtype_t w_dtype;  /* norm weights: FP32 or == dtype */
  int batch, seqlen, heads_q, heads_k, head_dim;
  int rotary_dim, interleaved, norm, max_pos;
  float eps;
  int64_t stride_q[3], stride_k[3];       /* {batch, token, head}, in elements */
  int64_t stride_qo[3], stride_ko[3];     /* q_out, k_out; backward: dq, dk */
  int64_t stride_dqo[3], stride_dko[3];   /* backward: gradients of q_out, k_out */
} attn_qk_params_t;
attn_status_t attn_qk_norm_rope(const attn_qk_params_t* p, const void* q, const void* k,
                                const void* w_q, const void* w_k, const float* cos,
                                const float* sin, const int32_t* positions, void* q_out,
                                void* k_out, int32_t* status, attn_stream_t stream);
/*
 * Its gradient, from q, k and the gradients of q_out, k_out: dq, dk (dtype) and
 * the weights' dw_q, dw_k (FP32 [head_dim], summed over all tokens and heads,
 * overwritten; NULL where not wanted).  Rows at negative positions get no
 * gradient (dq, dk untouched there) and add nothing to dw.  The order of the
 * sums is fixed: bitwise reproducible.  dq may be written over the gradient of
 * q_out (same strides), not over q.  workspace: 256-byte aligned,
 * attn_qk_norm_rope_bwd_workspace_size(p) bytes (of the current device).
 */
size_t attn_qk_norm_rope_bwd_workspace_size(const attn_qk_params_t* p);
attn_status_t attn_qk_norm_rope_bwd(const attn_qk_params_t* p, const void* q, const void* k,
                                    const void* w_q, const void* w_k, const float* cos,
                                    const float* sin, const int32_t* positions,
                                    const void* dq_out, const void* dk_out, void* dq, void* dk,
                                    float* dw_q, float* dw_k, void* workspace,
                                    size_t workspace_bytes, int32_t* status,
                                    attn_stream_t stream);

/*
 * Where the new tokens of a step go.  Request b holds context[b] tokens and
 * gets fresh[b] more; its page table is row b of block_table (int32,
 * [batch][cols], rows table_stride apart; page_size tokens a page).
 *   cu_seqlens [batch+1]: prefix sums of fresh;  seq_lens [batch]: context + fresh
 *   positions, slots [rows]: of the new tokens, packed in order of the requests
 *     (slot = page * page_size + position % page_size); rows past the last token are -1
 * With free_pages (int32 [n_free]) the pages that the new tokens need beyond
 * those held, ceil((context + fresh) / page_size) - ceil(context / page_size)
 * a request, are taken in order from free_pages[free_head[0] ..], written into
 * block_table, and free_head_out[0] = free_head[0] + pages taken; an empty list is
 * any address with n_free = 0.  With free_pages NULL the table is only read (a map
 * of tokens that have pages already) and free_head, free_head_out are ignored.
 * Out of range (status word): lengths that are negative or longer than cols *
 * page_size (the request counts as empty), more tokens than rows (the rest is
 * left out), pages outside [0, num_pages) or past n_free (slot -1, table entry -1).
 * The inputs are not changed (block_table apart), so a call can be repeated.
 * No output may overlap an input or another output.  batch <= 8192; page_size a power of two, 16 to
 * 256; cols * page_size <= 2^30; num_pages * page_size < 2^31.
 */
typedef struct {
  int batch, cols, page_size, num_pages, rows, n_free;
  int64_t table_stride;
} attn_kv_plan_params_t;
attn_status_t attn_kv_plan(const attn_kv_plan_params_t* p, const int32_t* context,
                           const int32_t* fresh, int32_t* block_table,
                           const int32_t* free_pages, const int32_t* free_head,
                           int32_t* cu_seqlens, int32_t* seq_lens, int32_t* positions,
                           int32_t* slots, int32_t* free_head_out, int32_t* status,
                           attn_stream_t stream);

/*
 * A cache of keys and values in 4 bits.  For a row x (one token, one kv head)
 * and each 32 neighbouring elements of it:
 *     s = bf16(max|x| / 7),  code = clamp(round(x / s), -7, 7) + 8,  value = (code - 8) s
 * (round to nearest, ties to even; s = 0: codes 8).  A group that holds an
 * infinity or a NaN reads back as NaN.  Arrays, contiguous and 16-byte aligned,
 * G = d / 32:
 *     codes  [num_pages][heads_kv][page_size][d / 2] bytes
 *     scales [num_pages][heads_kv][page_size][G]     bf16
 * A K row is 4 G words: word c G + g holds dims 32 g + 8 c .. + 7; a V row is
 * 8 G half-words: half-word r G + g holds dims 32 g + 4 r .. + 3; lowest
 * nibble first (the order in which attn_kv_decode reads them).
 * (d_qk, d_v): (64,64) (128,128) (192,128) (256,256).  page_size a power of
 * two, 16 to 256; num_pages * page_size < 2^31.
 */
typedef struct {
  void* k_codes;
  void* k_scales;
  void* v_codes;
  void* v_scales;
  int num_pages, page_size, heads_kv, d_qk, d_v;
} attn_kv4_cache_t;

/*
 * Rows into the cache and back.  k [tokens][heads_kv][d_qk], v
 * [tokens][heads_kv][d_v] of dtype (BF16 or FP16), strides {token, head} in
 * elements (multiples of 8), 16-byte aligned.  Token t lives at slots[t] (page *
 * page_size + offset); a negative slot leaves token t out (write: nothing is
 * stored; read: its row stays as it was); one past the cache does too, and sets
 * the status word.  A write's slots must differ from each other: of rows
 * written to one slot in one call, parts of either may remain.
 * Values are rounded once to dtype when read.
 */
attn_status_t attn_kv_write(const attn_kv4_cache_t* cache, attn_dtype_t dtype, int tokens,
                             const void* k, const int64_t stride_k[2], const void* v,
                             const int64_t stride_v[2], const int32_t* slots, int32_t* status,
                             attn_stream_t stream);
attn_status_t attn_kv_read(const attn_kv4_cache_t* cache, attn_dtype_t dtype, int tokens,
                            void* k, const int64_t stride_k[2], void* v,
                            const int64_t stride_v[2], const int32_t* slots, int32_t* status,
                            attn_stream_t stream);

/*
 * Attention of the last seqlen_q tokens of each sequence (1 to 256: a decode
 * step, drafted tokens, a short chunk) over the 4-bit cache.  (It reads the cache
 * once for every 16 query rows a kv head, 8 at d_v = 256: from about 100 rows on,
 * attn_kv_read and attn_fwd are quicker.)  Sequence b holds
 * seq_lens[b] tokens, those seqlen_q among them, in the pages of row b of
 * block_table.  Query i stands at pos = seq_lens[b] - seqlen_q + i and sees
 * tokens j <= pos with window_left < 0, or j >= pos - window_left, or
 * j < sinks (a sliding window whose first tokens stay visible).
 *     o   [batch][seqlen_q][heads_q][d_v] of o_dtype, lse FP32 [batch][heads_q][seqlen_q]
 * (natural log; a query that sees nothing, of an empty sequence or at a
 * negative position, gets O = 0, LSE = -inf).  Entries of the table past a
 * sequence's last page, entries of pages that no query sees a token of (behind
 * the window: such pages may be given away), and what a page holds past its last
 * token, are not looked at.  Sums are FP32.  A bf16 q row enters the first
 * product in FP16, times a power of two that keeps all but elements 2^27 times
 * smaller than its largest; probabilities times V's scales are rounded to FP16, in
 * units set by the largest V scale, of any group of dims, of the tokens met so far:
 * beside a V scale 2^24 times the others', the others lose bits.  So O carries an
 * error of up to 2^-11 of sum p |v|, with an FP32 output as with a 16-bit one.  V
 * scales of 2^101 and more (values above 10^30) may give infinities, and so may scores
 * of 2^22 and more (FP32 tells those in the exponentials no better than 1/4).  The result
 * does not depend on other sequences' lengths beyond the order of its sums, and is
 * bitwise reproducible for the same call on the same device.
 * Lengths are read on the device: a captured call serves any lengths.
 * seq_lens out of [0, cols * page_size] count as 0 and set the status word; so
 * does a page outside the cache (that sequence's result is then undefined).
 * workspace: 256-byte aligned, attn_kv_decode_workspace_size() bytes (of the
 * current device); it needs no preparation, and calls that may overlap in
 * time need one each.
 */
typedef struct {
  attn_dtype_t dtype;    /* q: BF16 or FP16 */
  attn_dtype_t o_dtype;  /* == dtype, or FP32: the sums as they are (probabilities have 11 bits) */
  int batch, seqlen_q, heads_q;  /* heads_q % heads_kv == 0, heads_q / heads_kv <= 128 */
  int64_t stride_q[3], stride_o[3]; /* {batch, token, head} */
  int cols;              /* columns of block_table; cols * page_size <= 2^30 */
  int64_t table_stride;  /* elements between its rows */
  int window_left, sinks;
  float softmax_scale;
} attn_kv4_decode_params_t;
size_t attn_kv_decode_workspace_size(const attn_kv4_decode_params_t* p,
                                      const attn_kv4_cache_t* cache);
attn_status_t attn_kv_decode(const attn_kv4_decode_params_t* p, const attn_kv4_cache_t* cache,
                              const void* q, const int32_t* block_table,
                              const int32_t* seq_lens, void* o, float* lse, void* workspace,
                              size_t workspace_bytes, int32_t* status, attn_stream_t stream);

/*
 * attn_kv_decode for batches whose requests share their first tokens (a system prompt,
 * a document, samples of one request): the same results, to rounding, but what a
 * group's requests share is read and converted once for all of them, and multiplied
 * with all their query rows at a time.  (On a GB300 that pays where attn_kv_decode would read
 * 300 MB of shared codes and scales over and over, say 16 requests over 16K tokens of 8 kv heads of
 * 128, and costs 10 to 30 us more than attn_kv_decode for few requests or short prefixes.)
 * Requests group_starts[g] .. group_starts[g + 1] - 1 are group g (int32 [groups + 1],
 * ascending; requests outside all groups share nothing), and the first shared_lens[g]
 * tokens of each of them lie in the same pages: their rows of block_table name the same
 * pages there, which the call relies on and does not check.  A prefix counts in whole
 * multiples of 64 tokens; the rest of it is read as each request's own.  A request that
 * has fewer tokens than the prefix and the seqlen_q newest shares nothing, and neither
 * does a group with fewer than two that do.
 * p as in attn_kv_decode, without a window (window_left = -1; sinks is ignored).  Of the
 * shared part, codes times scales are FP16 operands: exact, but elements of K whose scale is
 * below 2^-28 of the largest one S_k of the 32 tokens around them are off by up to 2^-32 S_k.
 * Probabilities are rounded to FP16, in units that the row's largest product of a probability
 * and a V scale sets (the largest of each in any 32 tokens): O carries an error of up to 2^-11
 * of sum p |v|, as attn_kv_decode's does, and for each token one of up to 2^-31 of that
 * product.
 * group_starts that do not ascend within [0, batch] (no group shares anything then),
 * shared_lens out of [0, cols * page_size] (that group shares nothing) set the status
 * word, beside what attn_kv_decode reports.  Every wait of the kernels on an mbarrier has a
 * limit (2 s); when one runs out the status word tells ATTN_ERR_TIMEOUT, and rows of O and LSE
 * that lack a part for it are NaN.
 * Bitwise reproducible for the same call on the same device.  Lengths, groups and prefixes
 * are read on the device: a captured call serves any.
 * workspace: 256-byte aligned, attn_kv_decode_shared_workspace_size() bytes (of the
 * current device); it needs no preparation, and calls that may overlap in time need
 * one each.
 */
size_t attn_kv_decode_shared_workspace_size(const attn_kv4_decode_params_t* p,
                                            const attn_kv4_cache_t* cache, int groups);
attn_status_t attn_kv_decode_shared(const attn_kv4_decode_params_t* p,
                                    const attn_kv4_cache_t* cache, int groups,
                                    const int32_t* group_starts, const int32_t* shared_lens,
                                    const void* q, const int32_t* block_table,
                                    const int32_t* seq_lens, void* o, float* lse,
                                    void* workspace, size_t workspace_bytes, int32_t* status,
                                    attn_stream_t stream);

/*
 * The attention weights that cached tokens receive from the last seqlen_q tokens of
 * each sequence, from the log-sum-exp of those tokens' attention over this cache (lse
 * as attn_kv_decode writes it, with the same scale, window and first tokens):
 *     weights[b][h][j] (+)= sum over i < seqlen_q and the query heads a of kv head h
 *                           of exp(softmax_scale q[b][i][a] k[b][h][j] - lse[b][a][i])
 * over the queries i that see token j.  FP32, tokens contiguous, {batch, head} strides
 * stride_w, `capacity` entries a row.  accumulate = 1: entries of tokens that were
 * there before (j < seq_lens[b] - seqlen_q) are added to, those of the seqlen_q
 * newest are set; entries of tokens that no query sees stay.  accumulate = 0: the
 * entries of all seq_lens[b] tokens are set (to 0 where no query sees them; with seqlen_q = 0
 * all of them are, and q and lse are not looked at).  Entries from seq_lens[b] on are not
 * touched.  What table entries and page contents are not looked at, is as in
 * attn_kv_decode.  Scores are those of attn_kv_decode, to rounding; sums are FP32 in
 * an order that does not depend on the other sequences: bitwise reproducible.
 * seq_lens out of [0, min(cols * page_size, capacity)] count as 0 and set the status
 * word; so does a page outside the cache that holds a visible token (that sequence's
 * entries are then undefined).
 */
typedef struct {
  attn_dtype_t dtype;    /* q: BF16 or FP16 */
  int batch, seqlen_q, heads_q;  /* as in attn_kv_decode */
  int64_t stride_q[3];   /* {batch, token, head} */
  int cols;
  int64_t table_stride;
  int window_left, sinks;
  float softmax_scale;
  int accumulate;
  int capacity;          /* entries of a row of weights */
  int64_t stride_w[2];   /* {batch, head}, in elements; rows must not overlap */
} attn_kv4_weights_params_t;
attn_status_t attn_kv_weights(const attn_kv4_weights_params_t* p, const attn_kv4_cache_t* cache,
                              const void* q, const int32_t* block_table, const int32_t* seq_lens,
                              const float* lse, float* weights, int32_t* status,
                              attn_stream_t stream);

/*
 * Eviction: each sequence of more than `keep` tokens is cut down to that many, each kv
 * head by itself.  Of n = seq_lens[b] tokens there stay the first f = min(first[b],
 * keep) (first NULL: none), the last r = min(recent, keep - f) and, of those
 * between, the keep - f - r with the largest weight; of equal ones those with the lower
 * index; NaN lies below all numbers.  They keep their order: row i of a kept sequence
 * is what row kept[b][h][i] was, codes, scales and weight.
 *     kept         int32 [batch][heads_kv][keep], contiguous; -1 past the tokens held
 *     seq_lens_out int32 [batch]: min(seq_lens, keep)
 *     weights_out  FP32, strides {batch, head} stride_wo; may be `weights` itself (same
 *                  strides).  Entries past the tokens held are not touched.
 * The keys of the cache are rotated already, so attention over what stays is attention
 * over those tokens; positions of later tokens are the caller's (plan's, plus what was
 * evicted).  Rows in front of the first evicted token are not written: a prefix that
 * other sequences share may stay in front under `first`.  Pages that hold other tokens
 * of an evicted sequence must be its own.
 * With free_head the pages of evicted sequences that hold neither one of the `keep` tokens
 * nor a first one (columns from ceil(max(keep, first[b]) / page_size) on) go back to the list
 * that attn_kv_plan takes from: with g of them in all, free_pages[free_head[0] - g ..
 * free_head[0]) is written, sequence after sequence, and free_head_out[0] =
 * free_head[0] - g.  (Where first[b] > keep, a budget shorter than what it protects, pages
 * of the first tokens that go are the caller's to give back once, since other sequences may
 * hold them; and unless keep is a multiple of page_size the sequence ends inside such a page,
 * in which attn_kv_plan would put its next tokens: if others hold it, the caller
 * gives the sequence a copy of that page before.)  If there are not g entries in front of free_head[0], or that lies
 * past n_free, no page is given back, free_head_out[0] = free_head[0] and the status word
 * is set.  A page outside the cache is given back as -1 and sets the status word, as one
 * that holds a row to move does (that row then stays).  free_head NULL: free_pages and
 * free_head_out are ignored.
 * block_table is not changed: its entries past the tokens held are not looked at by
 * the other calls, and attn_kv_plan writes them again.
 * seq_lens out of [0, min(cols * page_size, capacity)] count as 0 and set the status
 * word.  Nothing depends on the order in which blocks run.  batch * heads_kv <= 2^24, with a
 * free list batch <= 2^16.
 */
typedef struct {
  int batch, cols;
  int64_t table_stride;
  int keep, recent;      /* keep >= 1, recent >= 0 */
  int capacity;          /* entries of a row of weights and weights_out */
  int64_t stride_w[2], stride_wo[2];
  int n_free;            /* entries of free_pages */
} attn_kv4_evict_params_t;
attn_status_t attn_kv_evict(const attn_kv4_evict_params_t* p, const attn_kv4_cache_t* cache,
                            const int32_t* block_table, const int32_t* seq_lens,
                            const int32_t* first, const float* weights, float* weights_out,
                            int32_t* kept, int32_t* seq_lens_out, int32_t* free_pages,
                            const int32_t* free_head, int32_t* free_head_out, int32_t* status,
                            attn_stream_t stream);

/* Synchronises `stream` and returns the status word in `workspace`
 * (ATTN_OK, ATTN_ERR_BAD_METADATA, ATTN_ERR_TIMEOUT or, for the head-dim-512
 * backward, ATTN_ERR_WORKSPACE). */
attn_status_t attn_query_status(const void* workspace, attn_stream_t stream);

/* Message of the last error returned on this thread ("" if none). */
const char* attn_last_error(void);

/* Number of kernels the last successful attn_fwd / attn_bwd / attn_lse_merge
 * call on this thread enqueued. */
int attn_last_launch_count(void);

/*
 * TEST ONLY: fault injection for the bounded-wait unwind path.  Every wait of
 * the attention kernels on an mbarrier phase has a wall-clock limit (2 s by
 * default); when one runs out the CTA raises ATTN_ERR_TIMEOUT in the status
 * word, lets its in-flight copies land, drains its MMAs, frees its TMEM and
 * returns -- no kernel traps or hangs (PR #3699's bot review found a
 * "missing wait" on a reused barrier phase; this is the guard against that
 * class of bug).  This call arms the NEXT attn_fwd / attn_bwd* /
 * attn_kv_decode_shared call on the calling thread, then clears itself: in every kernel selected by
 * `kernel_mask` (ATTN_DEBUG_* bits), one CTA leaves out load number
 * `drop_load` (-1: none) and, if `wait_limit_ns` is non-zero, waits at most
 * that long instead of 2 s.  In the dQ kernel, which runs work items from a
 * queue, it is the CTA that runs the first work item (the heaviest query
 * tile of the first head), the load is the K tile number `drop_load` of that
 * item, and every CTA of the launch uses the shorter limit (a healthy wait
 * lasts microseconds); in the other
 * kernels it is the first CTA (block 0,0,0), the load number counts its
 * stage/ring loads (in the shared prefix's kernel the K tiles that it converts),
 * and only that CTA uses the shorter limit.  No other call
 * is affected.  A dropped load makes a wait run out, so the call reports
 * ATTN_ERR_TIMEOUT through attn_query_status and leaves its outputs
 * undefined (attn_kv_decode_shared: as stated there); the device stays usable and later calls are unaffected.
 */
enum {
  ATTN_DEBUG_FWD = 1,    /* forward kernel */
  ATTN_DEBUG_DQ = 2,     /* dQ kernel, or the dQ GEMM of the materialising backward */
  ATTN_DEBUG_DKDV = 4,   /* dK/dV kernel, or the dK/dV GEMMs of the materialising backward */
  ATTN_DEBUG_SCORES = 8, /* P/dS scores kernel of the materialising backward */
  ATTN_DEBUG_SHARED = 16 /* prefix kernel of attn_kv_decode_shared */
};
void attn_debug_inject(unsigned kernel_mask, int drop_load, uint64_t wait_limit_ns);

#ifdef __cplusplus
}
#endif
#endif /* ATTN_H_ */
