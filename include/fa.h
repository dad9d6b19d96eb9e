/*
 * fa.h -- C ABI of the B200 (sm_100a) exact attention library
 *         (libfa.so).
 *
 * The operation: O = softmax(scale * Q K^T + mask) V for every (batch, head),
 * computed tile by tile with the online softmax, never writing the L_q x L_k
 * score matrix to memory, plus the per-row log-sum-exp of the scaled, masked
 * scores.
 *   - formulas: "PyTorch Transformer Flash Attention机制" section 1;
 *     "FlashAttention算法原理与性能优化实战" section 1.1;
 *   - online softmax: "Flash Attention是怎么做到又快又省显存的？" (Online
 *     normalizer derivation) and "FlashAttention算法原理与性能优化实战"
 *     section 1.2.2;
 *   - operator statement (4-D [B,H,S,D] inputs, output shaped like the query,
 *     fp32 softmax statistics of shape [B,H,S], scale_value, pre_tokens /
 *     next_tokens window): "FlashAttention算法原理与性能优化实战" section 2.2;
 *   - logsumexp kept for the backward pass: Triton FA2 walkthrough;
 *   - MQA/GQA and the causal mask: "FlashAttention算法原理与性能优化实战"
 *     section 1.3.
 *
 * All functions return 0 (FA_OK) or a negative fa_status; none aborts.
 * Every pointer argument marked "device" must point to memory the current
 * CUDA device can read/write; the library allocates no memory and keeps no
 * state between calls other than one device-side status word and the
 * static scratch of fa_fwd_splitkv_static (module memory, not allocated by
 * any call).
 */
#ifndef FA_H
#define FA_H

#include <stddef.h>
#include <cuda_runtime.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FA_F16 = 0,  /* IEEE binary16 */
    FA_BF16 = 1  /* bfloat16 */
} fa_dtype;

typedef enum {
    FA_MASK_NONE = 0,
    FA_MASK_BOOL = 1,   /* uint8; nonzero hides the key */
    FA_MASK_F16 = 2,    /* IEEE binary16, added to the scaled score */
    FA_MASK_F32 = 3     /* binary32, added to the scaled score */
} fa_mask_type;

typedef enum {
    FA_OK = 0,
    FA_ERR_NULL = -1,     /* q or out is NULL while L_q > 0, or k or v is
                             NULL while L_k > 0 */
    FA_ERR_SHAPE = -2,    /* B, H, H_kv < 1; L_q, L_k < 0; H % H_kv != 0;
                             or a size whose byte extent overflows */
    FA_ERR_HEADDIM = -3,  /* D not supported: the 16-bit forward entries take
                             any multiple of 16 in [16, 128]; fa_fwd_fp8
                             takes 32, 64, 128 */
    FA_ERR_DTYPE = -4,    /* dtype not FA_F16 / FA_BF16 */
    FA_ERR_ALIGN = -5,    /* q, k, v, out not 16-byte aligned, or lse not
                             4-byte aligned */
    FA_ERR_ARG = -6,      /* scale is negative, NaN or infinite */
    FA_ERR_CUDA = -7,     /* a CUDA runtime/driver call failed (launch,
                             tensor-map encoding, device query) */
    FA_ERR_TIMEOUT = -8,  /* a device-side wait gave up (watchdog); the
                             outputs of that launch are not valid */
    FA_ERR_WORKSPACE = -9, /* workspace smaller than the size the matching
                              *_workspace_bytes() call returns */
    FA_ERR_SCRATCH = -10   /* fa_fwd_splitkv_static: the problem needs more
                              than FA_STATIC_SCRATCH_BYTES of scratch */
} fa_status;

/*
 * fa_fwd -- exact attention forward on `stream` (asynchronous).
 *
 *   q     device, [B, H,    L_q, D] contiguous, element type `dtype`
 *   k, v  device, [B, H_kv, L_k, D] contiguous, element type `dtype`
 *   out   device, [B, H,    L_q, D] contiguous, element type `dtype`
 *         (written; RNE rounding of the fp32 result)
 *   lse   device, [B, H, L_q] contiguous fp32, or NULL to skip it.
 *         lse = ln(sum_j exp(scale * q_i . k_j)) over the visible keys j;
 *         -inf for a row with no visible key (whose out row is 0).
 *   scale finite, >= 0 (the pages use 1/sqrt(D); this ABI has no default).
 *   causal, window_left, window_right:
 *         key j is visible from query i iff j < L_k and
 *         (window_left  < 0 or j >= i - window_left) and
 *         (window_right < 0 or j <= i + window_right) and
 *         (causal == 0 or j <= i).  Indices are raw positions (row i of Q
 *         and row j of K), so causal == 1 equals window_right = 0.
 *         A negative window means unbounded (the pages' INT_MAX default).
 *   GQA / MQA: query head h reads key/value head h / (H / H_kv).
 *   L_q == 0 is a no-op; L_k == 0 writes out = 0 and lse = -inf.  A
 *   pointer to a tensor with no elements may be NULL.
 *
 * Buffers are owned by the caller and must not overlap out/lse with inputs.
 * The call only enqueues work: argument errors are returned before anything
 * is enqueued; device-side watchdog errors are reported by
 * fa_get_device_status().
 *
 * Decoding shapes -- at most two query rows per K/V head (L_q * H / H_kv
 * <= 2) and D in {16, 32, 64, 128} -- run on a CUDA-core kernel that
 * streams the key/value cache through shared memory (the product with one
 * or two query rows is a matrix-vector product, far from the tensor cores'
 * work); it keeps the softmax weights in fp32.  Everything else runs on the
 * tcgen05 tensor-core kernel.  The result is the same function either way.
 */
int fa_fwd(const void *q, const void *k, const void *v, void *out, float *lse,
           int B, int H, int H_kv, int L_q, int L_k, int D, float scale,
           int causal, int window_left, int window_right, int dtype,
           cudaStream_t stream);

/*
 * fa_fwd_ex -- fa_fwd with the optional inputs and outputs of the operator
 * statement in "FlashAttention算法原理与性能优化实战" §2.2: an attention mask
 * and the two softmax statistics kept for the backward pass.
 *
 *   mask, mask_type  device, or NULL with FA_MASK_NONE.  Element
 *               (b, h, i, j) is mask[b*mask_stride_b + h*mask_stride_h +
 *               i*mask_stride_q + j] (strides in elements, >= 0; a stride
 *               of 0 broadcasts, e.g. [L_q, L_k] for every batch and head:
 *               0, 0, L_k).  FA_MASK_BOOL: a nonzero byte hides key j from
 *               query i.  FA_MASK_F16 / FA_MASK_F32: the value is added to
 *               scale * q_i . k_j before the softmax (-inf hides).  The
 *               causal / window rule applies on top.  The caller guarantees
 *               every addressed element lies in the buffer.  16-byte
 *               aligned base and strides take the vectorised load path.
 *   softmax_max, softmax_sum  device [B, H, L_q] fp32, both or neither
 *               (NULL): the row max m_i of the scaled, masked scores and
 *               sum_j exp(s_ij - m_i); lse = m + ln(sum).  A row with no
 *               visible key gets -inf and 0.
 * Other arguments, errors and edge cases as fa_fwd; FA_ERR_ARG for a bad
 * mask_type or a negative stride.
 */
int fa_fwd_ex(const void *q, const void *k, const void *v, void *out, float *lse,
              float *softmax_max, float *softmax_sum, const void *mask, int mask_type,
              long long mask_stride_b, long long mask_stride_h, long long mask_stride_q,
              int B, int H, int H_kv, int L_q, int L_k, int D, float scale, int causal,
              int window_left, int window_right, int dtype, cudaStream_t stream);

/*
 * fa_fwd_fp8 -- exact attention forward on fp8 (E4M3) inputs.  The pages
 * list fp8 among FlashAttention-2's input types ("PyTorch Transformer Flash
 * Attention机制" §5) without details; this entry reads them as: q, k, v hold
 * E4M3 codes (OCP "fn" encoding: bias 7, no infinities, largest 448) whose
 * real values are code * descale_{q,k,v}; the scores are
 * scale * descale_q * descale_k * (q_i . k_j) accumulated in fp32; P enters
 * the P.V product rounded to E4M3 (the tensor cores' fp8 kind takes both
 * operands in 8 bits) while the normaliser sums the unrounded fp32 weights;
 * O = descale_v * P.V / l is written as bf16.
 *
 *   q         device, [B, H,    L_q, D] E4M3 codes (1 byte each)
 *   k, v      device, [B, H_kv, L_k, D] E4M3 codes
 *   out       device, [B, H,    L_q, D] bfloat16 (written)
 *   lse       device, [B, H, L_q] fp32 or NULL (natural log, as fa_fwd)
 *   descale_q, descale_k, descale_v  finite, >= 0 (1 = codes are the values)
 *   D in {32, 64, 128} (rows of at least 32 bytes), else FA_ERR_HEADDIM.
 * Masks, windows, GQA, edge cases and errors as fa_fwd.
 */
int fa_fwd_fp8(const void *q, const void *k, const void *v, void *out, float *lse, int B,
               int H, int H_kv, int L_q, int L_k, int D, float scale, float descale_q,
               float descale_k, float descale_v, int causal, int window_left,
               int window_right, cudaStream_t stream);

/*
 * fa_fwd_host_workspace_bytes -- bytes of device workspace fa_fwd_host
 * needs (0 if the sizes are invalid): two slots, each holding one chunk's
 * q, k, v, out and lse.
 */
size_t fa_fwd_host_workspace_bytes(int B, int H, int H_kv, int L_q, int L_k, int D,
                                   int n_chunks);

/*
 * fa_fwd_host -- fa_fwd on HOST buffers (pinned memory lets the copies run
 * asynchronously and overlap; pageable memory works but serialises them).
 * The B*H_kv key/value heads (with their query heads) are cut into
 * n_chunks contiguous ranges; chunk c's q, k, v are copied in on a copy
 * stream, its forward runs on `stream`, its out and lse are copied back on
 * a second copy stream, each chunk through one of two device slots in
 * `workspace`, so the copies in both directions overlap the kernels of
 * neighbouring chunks.  Arguments as fa_fwd except:
 *   q, k, v, out, lse  HOST pointers, same layouts (lse may be NULL)
 *   workspace          device, 256-byte aligned, at least
 *                      fa_fwd_host_workspace_bytes(...) bytes
 *   n_chunks           >= 1 (FA_ERR_ARG otherwise)
 * Returns after enqueueing; `stream` is ordered after the last copy out, so
 * synchronising it makes out and lse valid.  The copy streams and events
 * are created by the first call on each device (make it before any stream
 * capture); calls on one device must not overlap.
 */
int fa_fwd_host(const void *q, const void *k, const void *v, void *out, float *lse, int B,
                int H, int H_kv, int L_q, int L_k, int D, float scale, int causal,
                int window_left, int window_right, int dtype, void *workspace,
                size_t workspace_bytes, int n_chunks, cudaStream_t stream);

/*
 * fa_splitkv_workspace_bytes -- bytes of device workspace fa_fwd_splitkv
 * needs for these sizes (0 if the sizes are invalid): B*H*L_q*n_splits rows
 * of a D-wide fp32 partial output plus an (m, l) pair each.
 */
size_t fa_splitkv_workspace_bytes(int B, int H, int L_q, int D, int n_splits);

/*
 * fa_fwd_splitkv -- the same forward as fa_fwd, computed in n_splits
 * (1..64) slices of each query tile's key range: one launch writes every
 * slice's unnormalised output and (running max, normaliser) to `workspace`,
 * a second launch merges the slices of each row with the online-softmax
 * rescaling ("FlashAttention算法原理与性能优化实战" §1.2.2).  Meant for
 * shapes with few query tiles and long key ranges (decoding), where fa_fwd
 * would leave most SMs idle.  Arguments as fa_fwd, plus
 *   n_splits         number of key slices, 1..64 (FA_ERR_ARG otherwise)
 *   workspace        device, 256-byte aligned, caller-owned, at least
 *                    fa_splitkv_workspace_bytes(B, H, L_q, D, n_splits)
 *                    bytes (FA_ERR_WORKSPACE if smaller, FA_ERR_NULL if
 *                    NULL while L_q, L_k > 0); its contents on entry do not
 *                    matter and are overwritten.
 * Calls that share a workspace must not overlap on the GPU.
 */
int fa_fwd_splitkv(const void *q, const void *k, const void *v, void *out, float *lse,
                   int B, int H, int H_kv, int L_q, int L_k, int D, float scale,
                   int causal, int window_left, int window_right, int dtype,
                   int n_splits, void *workspace, size_t workspace_bytes,
                   cudaStream_t stream);

/*
 * fa_fwd_fp8_ex -- fa_fwd_fp8 with fa_fwd_ex's optional attention mask and
 * softmax statistics (same layouts and meaning; the mask's values are added
 * to the full-scale scores scale * descale_q * descale_k * q_i . k_j, and
 * softmax_max / softmax_sum refer to those scores).  Errors as fa_fwd_fp8
 * and fa_fwd_ex.
 */
int fa_fwd_fp8_ex(const void *q, const void *k, const void *v, void *out, float *lse,
                  float *softmax_max, float *softmax_sum, const void *mask, int mask_type,
                  long long mask_stride_b, long long mask_stride_h, long long mask_stride_q,
                  int B, int H, int H_kv, int L_q, int L_k, int D, float scale,
                  float descale_q, float descale_k, float descale_v, int causal,
                  int window_left, int window_right, cudaStream_t stream);

/*
 * fa_fwd_fp8_splitkv -- fa_fwd_fp8 computed in key slices as
 * fa_fwd_splitkv does (decoding over an fp8 key/value cache).  The slices'
 * partial outputs are fp32 in units of the V codes; the merge applies
 * descale_v and writes bf16.  Arguments as fa_fwd_fp8, plus n_splits,
 * workspace and workspace_bytes as fa_fwd_splitkv (the workspace size is
 * fa_splitkv_workspace_bytes(B, H, L_q, D, n_splits), the same as for
 * 16-bit inputs).  D must be 32, 64 or 128 (FA_ERR_HEADDIM otherwise).
 */
int fa_fwd_fp8_splitkv(const void *q, const void *k, const void *v, void *out, float *lse,
                       int B, int H, int H_kv, int L_q, int L_k, int D, float scale,
                       float descale_q, float descale_k, float descale_v, int causal,
                       int window_left, int window_right, int n_splits, void *workspace,
                       size_t workspace_bytes, cudaStream_t stream);

/*
 * fa_bwd_workspace_bytes -- bytes of device workspace fa_bwd needs (0 if
 * the sizes are invalid): an fp32 dQ accumulator [B, H, L_q, D] and two
 * fp32 row vectors [B, H, roundup(L_q, 128)].
 */
size_t fa_bwd_workspace_bytes(int B, int H, int L_q, int D);

/*
 * fa_bwd -- exact attention backward on `stream` (asynchronous): the
 * gradients of sum(dout .* out) for out = fa_fwd(q, k, v, ...), with the
 * attention matrix recomputed from q, k and the forward's lse instead of
 * stored ("FlashAttention算法原理与性能优化实战" §1.2.3, recomputation; the
 * Triton FA2 walkthrough keeps the logsumexp for the backward pass).  With
 * P = softmax(scale q k^T + mask):
 *     dv = P^T dout,  dS = P .* (dout v^T - delta),  delta_i = dout_i . out_i,
 *     dq = scale dS k,  dk = scale dS^T q,
 * and for GQA the query heads that share a key/value head add into it.
 *
 *   q, out, dout  device, [B, H,    L_q, D], element type `dtype`
 *   k, v          device, [B, H_kv, L_k, D], element type `dtype`
 *   lse           device, [B, H, L_q] fp32: the forward's lse (-inf rows
 *                 see no key and get dq = 0)
 *   dq            device, [B, H,    L_q, D] written (RNE of fp32)
 *   dk, dv        device, [B, H_kv, L_k, D] written
 *   scale, causal, window_left, window_right, dtype: as fa_fwd, and the
 *                 same values the forward used
 *   workspace     device, 256-byte aligned, caller-owned, at least
 *                 fa_bwd_workspace_bytes(B, H, L_q, D) bytes
 *                 (FA_ERR_WORKSPACE if smaller); contents on entry do not
 *                 matter.  Calls that share a workspace must not overlap.
 * L_q == 0 writes dk = dv = 0; L_k == 0 writes dq = 0.  Pointers to tensors
 * with no elements may be NULL.  q, k, v, out, dout, dq, dk, dv need
 * 16-byte alignment, lse 4 bytes (FA_ERR_ALIGN).  Errors as fa_fwd.
 */
int fa_bwd(const void *q, const void *k, const void *v, const void *out, const void *dout,
           const float *lse, void *dq, void *dk, void *dv, int B, int H, int H_kv, int L_q,
           int L_k, int D, float scale, int causal, int window_left, int window_right,
           int dtype, void *workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * fa_bwd_ex -- fa_bwd for a forward that used an attention mask (fa_fwd_ex):
 * P is recomputed with the same mask (same arguments, same reading: a
 * nonzero bool hides the key, a float is added to the scaled score; element
 * (b, h, i, j) at mask[b*mask_stride_b + h*mask_stride_h + i*mask_stride_q
 * + j]).  The mask itself gets no gradient.  Other arguments and errors as
 * fa_bwd; FA_ERR_ARG for a bad mask_type or a negative stride.
 */
int fa_bwd_ex(const void *q, const void *k, const void *v, const void *out, const void *dout,
              const float *lse, void *dq, void *dk, void *dv, const void *mask, int mask_type,
              long long mask_stride_b, long long mask_stride_h, long long mask_stride_q, int B,
              int H, int H_kv, int L_q, int L_k, int D, float scale, int causal,
              int window_left, int window_right, int dtype, void *workspace,
              size_t workspace_bytes, cudaStream_t stream);

/*
 * fa_splitkv_auto_splits -- the number of key slices the library would pick
 * for fa_fwd_splitkv / fa_fwd_fp8_splitkv on the current device (dtype:
 * FA_F16, FA_BF16, or 2 for E4M3 inputs).  For decoding shapes (at most two
 * query rows per K/V head: L_q * H / H_kv <= 2, head dims 16, 32, 64, 128)
 * the forward runs on the CUDA cores over a persistent grid of one CTA per
 * SM, and the slices make (B * H_kv * slices) work items whose last round is
 * nearly full; otherwise the tensor-core kernel's query tiles and slices
 * fill waves of one CTA per SM.  Returns 1 for empty or invalid sizes.
 * This is a planning helper: a split count, not a result of the method.
 */
int fa_splitkv_auto_splits(int B, int H, int H_kv, int L_q, int L_k, int D, int dtype);

/*
 * fa_fwd_splitkv_static -- fa_fwd_splitkv with no workspace argument: the
 * partials live in a fixed scratch array inside the library (static device
 * memory, FA_STATIC_SCRATCH_BYTES per device).  The pages have no
 * counterpart to this entry point; it exists for callers that cannot
 * allocate device memory at the time they run attention: a process whose
 * device memory is all owned by another allocator (so that a cudaMalloc
 * beside it could fail or fragment it), a serving loop that must not take
 * cudaMalloc's implicit device synchronisation and unbounded latency after
 * start-up, or a plug-in that has no handle on its host's allocator.  Every
 * call, and the library itself, allocates nothing.
 *
 * Arguments as fa_fwd_splitkv without `workspace` / `workspace_bytes`.
 * Returns FA_ERR_SCRATCH, before touching the GPU, when
 * fa_splitkv_workspace_bytes(B, H, L_q, D, n_splits) exceeds
 * FA_STATIC_SCRATCH_BYTES (16 MiB: e.g. 32768 query rows x n_splits at
 * D = 128; lower n_splits to fit); other errors as fa_fwd_splitkv.
 *
 * Set-up: the first call on each device (with that device current) looks
 * up the scratch's device address once and caches it, keyed on the device's
 * context (a context made anew, e.g. after cudaDeviceReset, is looked up
 * again on its first call); make that first call before any stream
 * capture.  Nothing in the scratch has to start at zero:
 * every partial the merge reads is written earlier in the same call.
 * There is ONE scratch per device: calls whose work overlaps on the GPU
 * (different streams, or different host threads) race on it and corrupt
 * each other's results; serialise them (one stream, or events).
 */
#define FA_STATIC_SCRATCH_BYTES ((size_t)16 << 20)
int fa_fwd_splitkv_static(const void *q, const void *k, const void *v, void *out,
                          float *lse, int B, int H, int H_kv, int L_q, int L_k, int D,
                          float scale, int causal, int window_left, int window_right,
                          int dtype, int n_splits, cudaStream_t stream);

/*
 * ---------------------------------------------------------------- serving
 * The entries below run one step of a serving engine around the attention:
 * fa_paged_plan builds the step's page tables from the request lengths,
 * fa_qk_norm_rope normalises and rotates q and k and writes k and v into
 * the paged cache, fa_fwd_paged attends over it.  fa_qk_norm_rope also has
 * the layouts that fa_fwd / fa_bwd train with, and fa_qk_norm_rope_bwd is
 * its gradient.  The pages have no counterpart.
 *
 * The paged cache: num_pages pages of page_size tokens of H_kv heads of D
 * values.  Element (page, row, head, d) lies at page * cache_stride_page +
 * row * cache_stride_token + head * cache_stride_head + d (element strides,
 * multiples of 8; k and v have the same), so [page, token, head, D] and
 * [page, head, token, D] both fit.  Slot s is row s % page_size of page
 * s / page_size.  Token x of request b lies in slot
 * block_table[b * table_stride + x / page_size] * page_size + x % page_size.
 * fa_paged_plan and fa_qk_norm_rope take any page_size >= 1, fa_fwd_paged powers
 * of two from 16 on.
 */

/*
 * fa_paged_plan -- one step's page tables, in one launch.
 *
 *   q_lens, ctx_lens  device int [B]: new tokens of each request, and tokens
 *                it has in the cache already (negative: 0)
 *   block_table  device int [B, table_stride], its first max_pages columns:
 *                on entry the pages of the tokens in the cache; new entries
 *                are written behind them, the others stay
 *   free_pages   device int [n_free]: pages that are handed out, from index
 *                0, to request 0 first
 *   cu_q         device int [B + 1] written: 0 and the running sums of q_lens
 *   kv_lens      device int [B] written: ctx_lens + q_lens
 *   positions    device int [num_tokens] written: token cu_q[b] + i has
 *                position ctx_lens[b] + i; -1 behind the last request
 *   slots        device long long [num_tokens] written: the token's cache
 *                slot, or -1 (behind the last request, or no page)
 *   counts       device int [3] written: new tokens in all, pages taken,
 *                new tokens without a slot (the free list ran out, whose
 *                table entries get -1, in this call or an earlier one, or the
 *                table's columns)
 * num_tokens is the capacity of positions and slots: a padded batch of a
 * captured graph has more than the requests' tokens, and tokens beyond it
 * are not written.  What is written may not overlap anything else (the next
 * step's ctx_lens is a copy of kv_lens, or the other of two).  FA_ERR_ARG for
 * such an overlap, page_size < 1 or table_stride < max_pages; pointers to arrays with no elements may be NULL.
 */
int fa_paged_plan(const int *q_lens, const int *ctx_lens, int *block_table,
                  long long table_stride, const int *free_pages, int n_free, int B, int max_pages,
                  int page_size, int num_tokens, int *cu_q, int *kv_lens, int *positions,
                  long long *slots, int *counts, cudaStream_t stream);

/* Rows of heads: element (b, l, h, d) at ptr + b * stride_b + l * stride_l +
 * h * stride_h + d, element strides that are positive multiples of 8 (any
 * value for an axis of one element), ptr 16-byte aligned. */
typedef struct {
    void *ptr;
    long long stride_b, stride_l, stride_h;
} fa_rows;

typedef struct {
    fa_rows q, k, v;          /* [B, L, H, D], [B, L, H_kv, D], [B, L, H_kv, D] */
    fa_rows q_out, k_out;     /* as q, k; the backward: the gradients of the outputs */
    const void *q_weight;     /* [D] of `dtype`, 16-byte aligned; NULL: no norm */
    const void *k_weight;
    const float *cos_sin;     /* [max_pos, rot_dim]: rot_dim/2 cosines, then the sines */
    const void *positions;    /* int or long long; (b, l) at b * stride_b + l * stride_l */
    long long positions_stride_b, positions_stride_l;   /* any, 0 broadcasts */
    void *k_cache, *v_cache;  /* the paged cache, or NULL */
    long long cache_stride_page, cache_stride_token, cache_stride_head;
    const long long *slots;   /* [B * L] contiguous */
    int num_pages, page_size; /* page_size >= 1 */
    int positions_64;         /* 0: int, 1: long long */
    int B, L, H, H_kv, D;     /* H_kv may be 0 */
    int rot_dim;              /* multiple of 16, 0 .. D */
    int max_pos;              /* rows of cos_sin */
    int interleaved;          /* pairs (2i, 2i+1); 0: (i, i + rot_dim/2) */
    int dtype;
    float eps;                /* >= 0; less than 2^-126 counts as that, so a row of zeros gives zeros */
} fa_rope_args;

/*
 * fa_qk_norm_rope -- for every head x of q and k, in one pass:
 *     y = R(weight .* x / sqrt(mean(x^2) + eps)),
 * where R turns the first rot_dim values by the token's position p: the pair
 * (u, w) becomes (u cos - w sin, w cos + u sin) with row p of cos_sin.  All
 * in fp32, rounded once.  y goes to q_out / k_out and, with a cache, k's y
 * and v unchanged go to the token's slot (k_out may then be NULL).  q_out may
 * be q itself, k_out k itself; no other overlap.  No two tokens may have the
 * same slot.
 *
 * A token whose position is negative or >= max_pos is padding: nothing of it
 * is written, so cos_sin has to have a row for every position in use.  A token whose slot is negative or >= num_pages * page_size
 * writes no cache.  L == 0 is a no-op.
 * Errors: FA_ERR_ARG for a bad rot_dim, eps, page_size or num_pages;
 * FA_ERR_ALIGN for a misaligned pointer or stride; others as fa_fwd.
 */
int fa_qk_norm_rope(const fa_rope_args *args, cudaStream_t stream);

/* Workspace bytes of fa_qk_norm_rope_bwd on the current device (0 for an
 * unsupported D): one fp32 row of D per block. */
size_t fa_qk_norm_rope_bwd_workspace_bytes(int D);

/*
 * fa_qk_norm_rope_bwd -- the gradients of sum(q_out .* dq_out) + sum(k_out .*
 * dk_out) for the outputs of fa_qk_norm_rope: args->q and k are its inputs,
 * args->q_out and k_out hold dq_out and dk_out (read); v and the cache are
 * not used.  Written:
 *   dq, dk       as q, k (RNE of fp32); zero for padding tokens
 *   dq_weight, dk_weight  device fp32 [D], given exactly where the weight is:
 *                sum over all rows of R^T(dy) .* x / sqrt(mean(x^2) + eps),
 *                in a fixed order (the same bits every time on one device)
 *   workspace    device, 256-byte aligned, at least
 *                fa_qk_norm_rope_bwd_workspace_bytes(D) bytes; contents on
 *                entry do not matter; not needed without weights.  Calls that
 *                share a workspace must not overlap on the GPU.
 * dq may be dq_out itself (dk likewise); no other overlap.  L == 0 writes
 * zero weight gradients.
 */
int fa_qk_norm_rope_bwd(const fa_rope_args *args, fa_rows dq, fa_rows dk, float *dq_weight,
                        float *dk_weight, void *workspace, size_t workspace_bytes,
                        cudaStream_t stream);

/* Workspace bytes of fa_fwd_paged on the current device (0 for an
 * unsupported D): two partial tiles of 256 rows and a counter for each SM.
 * They do not depend on the batch. */
size_t fa_paged_workspace_bytes(int D);

/*
 * fa_fwd_paged -- exact attention of each request's new tokens over its
 * paged key/value cache, which holds the new tokens' keys and values too:
 * prefill chunks, single tokens (decoding) and mixtures, in one launch.
 *
 *   q         device, rows of `dtype`: token t, head h at t * q_stride_t +
 *             h * q_stride_h; request b's new tokens are cu_q[b] ..
 *             cu_q[b+1] - 1 of the total_q rows
 *   k_cache, v_cache, block_table  as above; entries of pages that hold no
 *             visible key are not used, and an entry that names no page
 *             reads as zeros
 *   cu_q, kv_lens  device int [B + 1], [B]: kv_lens[b] tokens are in the
 *             cache, the last cu_q[b+1] - cu_q[b] of them new
 *   out       device, as q with its own strides; lse [total_q, H] fp32 or NULL
 *   causal, window_left, window_right  as fa_fwd, with positions in the
 *             request: new token i is at kv_len - q_len + i, and key j is
 *             visible iff j < kv_len, j <= position + window_right (0 when
 *             causal), j >= position - window_left
 *   D         a multiple of 16 in [16, 128]; H / H_kv at most 128
 *   B         at most 2^24; requests without new tokens (the rest of a captured
 *             batch) are skipped
 *   page_size a power of two, at least 16 (FA_ERR_ARG)
 *   workspace device, 256-byte aligned, at least fa_paged_workspace_bytes(D)
 *             bytes; contents on entry do not matter.  Calls that share a
 *             workspace must not overlap on the GPU.
 * A row that sees no key gets out = 0 and lse = -inf.  Rows of q, out and
 * lse outside cu_q[0] .. cu_q[B] are neither read into a result nor written.
 * Cache rows behind kv_len may hold anything, NaN included; a key or value
 * that some query of a request's 2 * floor(128 / (H / H_kv)) neighbouring
 * tokens sees has to be finite to leave the others' results finite.
 * Weights: the products and the softmax statistics are fp32.  For the product
 * with v a weight is rounded to 16 bits, as in fa_fwd, and moves out by at most
 * half a step (bf16 2^-8, fp16 2^-11) of sum_j p_j |v_j| / l; where a request's
 * new tokens times H / H_kv are at most 8 (decoding) what the rounding took off is
 * summed too (2^-16, 2^-22), as fa_fwd's contiguous decoding keeps them in fp32.
 * The results do not depend on timing: the same bits for the same lengths.
 * Lengths live on the device and are not checked on the host.  New tokens
 * behind total_q have no rows and tokens behind max_pages * page_size no keys;
 * the others keep their positions (kv_len - q_len + i with the lengths given).
 * total_q == 0 is a no-op.  Other errors as fa_fwd.
 */
int fa_fwd_paged(const void *q, long long q_stride_t, long long q_stride_h, const void *k_cache,
                 const void *v_cache, long long cache_stride_page, long long cache_stride_token,
                 long long cache_stride_head, const int *block_table, long long table_stride,
                 const int *cu_q, const int *kv_lens, void *out, long long out_stride_t,
                 long long out_stride_h, float *lse, int total_q, int B, int H, int H_kv, int D,
                 int num_pages, int page_size, int max_pages, float scale, int causal,
                 int window_left, int window_right, int dtype, void *workspace,
                 size_t workspace_bytes, cudaStream_t stream);

/*
 * fa_get_device_status -- synchronise `stream`, then read and clear the
 * device status word that the kernels set when a bounded wait gives up.
 * Returns FA_OK, FA_ERR_TIMEOUT, or FA_ERR_CUDA if the synchronisation or
 * the read failed.
 */
int fa_get_device_status(cudaStream_t stream);

/*
 * fa_selftest_wait_timeout -- exercise the device-side watchdog that every
 * kernel of this library relies on.  The pages have no counterpart; this
 * entry point exists so that the failure path can be tested on a GPU
 * without faulting it.  It enqueues one CTA of two warps on `stream`:
 *   warp 0 waits on an mbarrier phase that completes (one arrival), then on
 *          one that nothing completes; that wait gives up after the
 *          library's wait limit (1 s), raises the CTA's abort flag and sets
 *          the device status word, and the warp returns;
 *   warp 1 sleeps 0.5 s, then waits on the same never-completed phase and
 *          must give up as soon as warp 0 raises the abort flag, before its
 *          own limit.
 * `result` (device memory, 6 ints, written by the kernel):
 *   [0] 1 if the completed wait returned success, [1] 1 if the abandoned
 *   wait returned success (expected 0), [2] the abort flag afterwards
 *   (expected 1), [3] warp 0's abandoned wait in ms (about 1000), [4] 1 if
 *   warp 1's wait returned success (expected 0), [5] warp 1's wait in ms
 *   (about 500).
 * The kernel occupies one SM for about 1 s.  Afterwards
 * fa_get_device_status(stream) returns FA_ERR_TIMEOUT once (and clears
 * it); the context stays usable.  Returns FA_ERR_NULL for a NULL result,
 * FA_ERR_CUDA if the launch fails, else FA_OK.
 */
int fa_selftest_wait_timeout(int *result, cudaStream_t stream);

/* fa_status_string -- a static, human-readable name for a status code. */
const char *fa_status_string(int status);

/*
 * fa_version -- library version as major*10000 + minor*100 + patch.
 */
int fa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FA_H */
