/*
 * fa.h -- C ABI of the GB300 (sm_103a) flash-attention forward library
 *         (libfa_gb300.so).
 *
 * Two operations:
 *
 *   fa_prefill_fwd  dense attention forward, O = softmax(scale * Q K^T + mask) V,
 *                   for bf16/fp16, head_dim 64 or 128, MHA or GQA, causal or
 *                   not, Sq != Sk allowed.
 *                   Defined by: "Dense flash-attention prefill (gfx950 / MI355X)"
 *                   (opening paragraph: forward-only, bf16/fp16, head_dim
 *                   64/128, MHA or GQA, causal) and tessera #90
 *                   "compiler-generated flash_attn fwd+bwd" (flash_attn forward
 *                   commit note: S = scale*Q@K^T, causal/ragged mask, online
 *                   softmax, O += P@V; Sq/Sk/scale/causal are runtime values).
 *
 *   fa_decode_fwd   single-token attention over a KV cache whose valid length
 *                   lives in device memory, split over the sequence and merged
 *                   with a log-sum-exp combine.
 *                   Defined by: rocm-libraries #13108 "minimal single-token
 *                   attention decode" (interface description: Sq=1, contiguous
 *                   token-major K/V cache, device INT32 valid length, O only;
 *                   review finding: unused cache capacity may hold NaN and must
 *                   not reach the output; split-KV named as the next step).
 *
 *   fa_prefill_fwd_lse, fa_decode_fwd_lse
 *                   the same operations, also writing each row's log-sum-exp
 *                   lse = log sum_j exp(scale * <q, k_j>) over its visible keys
 *                   (fp32, natural log; -inf for a row with no visible key).
 *                   It is the per-row statistic a backward pass recomputes P
 *                   from (tessera #90, flash-attention backward commit note:
 *                   the "_pre" kernel's logsumexp) and the one partial results
 *                   over key ranges are merged by; rocm-libraries #13108 lists
 *                   the LSE output among what its first decode milestone
 *                   leaves out.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Tensors are contiguous, row-major, in device memory (or memory the device
 *   can address), 16-byte aligned:
 *       q, o   : [B, Sq, Hq,  D]     (decode: Sq = 1)
 *       k, v   : [B, Sk, Hkv, D]     (decode: [B, cap, Hkv, D], token-major)
 *   Query head h reads K/V head h / (Hq / Hkv) (contiguous GQA groups).
 * - The caller owns and allocates every tensor, including o.  The library
 *   keeps no pointer after the call returns.
 * - Work is enqueued on `stream`; no call synchronises the host.  A status of
 *   FA_OK means the work was validated and enqueued; device-side failures
 *   (a pipeline wait that exceeded its time limit) are reported by
 *   fa_device_error().
 * - Arguments are validated before anything touches the GPU; invalid
 *   arguments return FA_ERR_INVALID_ARG and enqueue nothing.
 * - Empty problems (B == 0, Sq == 0 or Hq == 0) are valid and enqueue nothing.
 *   Rows with no visible key (Sk == 0, or causal rows i with i + Sk - Sq < 0)
 *   produce O = 0.
 */
#ifndef FA_GB300_H
#define FA_GB300_H

#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { FA_BF16 = 0, FA_FP16 = 1 } fa_dtype_t;

typedef enum {
  FA_OK = 0,
  FA_ERR_INVALID_ARG = 1,  /* bad pointer, size, head config or dtype         */
  FA_ERR_UNSUPPORTED = 2,  /* valid request this build does not implement     */
  FA_ERR_CUDA = 3,         /* a CUDA runtime/driver call or launch failed     */
  FA_ERR_TIMEOUT = 4,      /* a device-side pipeline wait hit its time limit  */
  FA_ERR_TOO_LARGE = 5,    /* request exceeds fa_decode_fwd_noalloc's scratch */
  FA_ERR_BOUNDS = 6        /* a device-side bounds check skipped an access     */
} fa_status_t;

/*
 * fa_prefill_fwd -- attention forward for a batch of full sequences.
 *
 *   q      [B, Sq, Hq, D]   bf16 or fp16 (dtype), read only
 *   k, v   [B, Sk, Hkv, D]  same dtype, read only
 *   o      [B, Sq, Hq, D]   same dtype, written (every element of every row)
 *   Hq % Hkv == 0; D in {64, 128}; Sq, Sk >= 0; B, Hq, Hkv >= 0.
 *   scale  multiplies Q K^T (any finite value, applied as passed).
 *   causal nonzero: row i sees keys j <= i + (Sk - Sq) (bottom-right aligned;
 *          equals the usual top-left mask when Sq == Sk).
 *   dtype  FA_BF16 or FA_FP16.
 *
 * Arithmetic: Q K^T and P V on the tensor cores with fp32 accumulation;
 * softmax in fp32 (exp2 domain); P rounded to the input dtype before P V;
 * O = (P V) / l rounded once to the output dtype (round to nearest even).
 *
 * Returns FA_OK, FA_ERR_INVALID_ARG (null/misaligned pointer, negative size,
 * Hq % Hkv != 0, D not 64/128, unknown dtype, non-finite scale),
 * or FA_ERR_CUDA (tensor-map encode, attribute or launch failure).
 */
int fa_prefill_fwd(const void* q, const void* k, const void* v, void* o,
                   int B, int Hq, int Hkv, int Sq, int Sk, int D,
                   float scale, int causal, int dtype, cudaStream_t stream);

/*
 * fa_prefill_fwd_lse -- fa_prefill_fwd that also writes
 *
 *   lse    [B, Hq, Sq]  fp32, 4-byte aligned, written:
 *          lse[b,h,i] = log sum_j exp(scale * <q[b,i,h], k[b,j,h/G]>) over the
 *          keys row i sees; -inf for a row that sees none.
 *
 * Everything else as fa_prefill_fwd; lse == NULL is FA_ERR_INVALID_ARG.
 */
int fa_prefill_fwd_lse(const void* q, const void* k, const void* v, void* o, float* lse,
                       int B, int Hq, int Hkv, int Sq, int Sk, int D,
                       float scale, int causal, int dtype, cudaStream_t stream);

/*
 * fa_prefill_varlen_fwd -- fa_prefill_fwd over a batch of packed sequences of
 * different lengths (the gfx950 prefill README's TODO list names this
 * follow-up: packed varlen with per-sequence persistent scheduling).
 *
 *   q, o           [total_q, Hq, D]   sequences packed back to back
 *   k, v           [total_k, Hkv, D]
 *   cu_seqlens_q   [B + 1] int32 in device memory: sequence b's query rows are
 *   cu_seqlens_k   [cu_seqlens_q[b], cu_seqlens_q[b+1]), its keys likewise.
 *                  Read by the kernel only.
 *   max_seqlen_q   >= every query length (bounds the work plan)
 *   lse            NULL, or [Hq, total_q] fp32 written with each row's
 *                  log-sum-exp (-inf for a row with no visible key)
 *
 * Causal masking is bottom-right per sequence: row i of sequence b sees keys
 * j <= i + (Sk_b - Sq_b).  Keys of the neighbouring packed sequence that share
 * a tile are masked like keys past Sk.
 *
 * Scheduling: a one-CTA planning kernel reads the offsets on the device and
 * lists each sequence's 256-row query blocks, largest K/V tile count first;
 * the persistent prefill CTAs then claim (block, query head) items from that
 * list as they become free, so short and long sequences of a batch share the
 * grid instead of serialising.  The plan and the work counter live in
 * stream-ordered scratch (B * ceil(max_seqlen_q / 256) * 32 + 16 bytes).
 * Offsets that are not
 * 0 <= cu[b] <= cu[b+1] <= total, or a query length above max_seqlen_q, make
 * that sequence's rows unwritten and set the bounds bit reported by
 * fa_device_error().  Other rules as fa_prefill_fwd.
 */
int fa_prefill_varlen_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                          const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                          int B, int Hq, int Hkv, int total_q, int total_k, int max_seqlen_q,
                          int D, float scale, int causal, int dtype, cudaStream_t stream);

/*
 * fa_decode_fwd -- one new query token per sequence against a KV cache.
 *
 *   q              [B, 1, Hq, D]      bf16, read only
 *   kcache, vcache [B, cap, Hkv, D]   bf16, token-major, read only
 *   valid_len_dev  one int32 in device memory: the number of valid tokens L,
 *                  shared by the batch.  It is read by the kernels only (never
 *                  by the host), so the call never synchronises.  L is
 *                  clamped to [0, cap]; L == 0 gives O = 0.
 *   o              [B, 1, Hq, D]      bf16, written
 *   Hq % Hkv == 0; D in {64, 128}; cap >= 0.
 *
 * Cache entries at token positions >= L may hold anything, NaN and Inf
 * included: they are never used in arithmetic (zeroed in shared memory before
 * any MMA and given probability zero).
 *
 * Scratch: the split partials (fp32) are allocated stream-ordered on `stream`
 * (cudaMallocAsync / cudaFreeAsync), so calls on different streams never share
 * scratch.  Two kernels are enqueued: the split kernel and the combine, each
 * launched as a programmatic dependent of the grid before it on the stream:
 * before its griddepcontrol.wait a kernel only initialises shared-memory
 * barriers and prefetches its tensor maps, so it reads nothing an earlier
 * kernel may still be writing.
 *
 * Returns FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED (dtype other than
 * bf16), or FA_ERR_CUDA.
 */
int fa_decode_fwd(const void* q, const void* kcache, const void* vcache,
                  const int32_t* valid_len_dev, void* o,
                  int B, int Hq, int Hkv, int cap, int D, float scale,
                  cudaStream_t stream);

/*
 * fa_decode_paged_fwd -- decode of Sq new tokens per sequence (Sq = 1: the
 * single-token step; Sq > 1: tokens proposed by speculative decoding) for a
 * batch of sequences with their own lengths, over a paged KV cache (the
 * decode PR's deferred items: batched shapes, several query tokens, and
 * non-contiguous KV storage).
 *
 *   q              [B, Sq, Hq, D]                   bf16, read only
 *   kpages, vpages [num_pages, page_size, Hkv, D]   bf16, read only
 *   page_table     [B, max_pages] int32, device: sequence b's tokens
 *                  [p*page_size, (p+1)*page_size) live in physical page
 *                  page_table[b][p]
 *   seqlens        [B] int32, device: sequence b's valid length L (including
 *                  its Sq new tokens, whose K/V are already in the cache),
 *                  clamped to [0, max_pages * page_size]
 *   o              [B, Sq, Hq, D]                   bf16, written
 *   lse            NULL, or [B, Sq, Hq] fp32 written with each row's
 *                  log-sum-exp
 *
 * New token s (0-based) sits at position L - Sq + s and sees the keys
 * [0, L - Sq + s] (bottom-right causal); rows that see no key give O = 0 and
 * lse = -inf.
 *   page_size      a positive multiple of 32
 *
 * Only the pages that hold a sequence's first seqlens[b] tokens are read; page
 * ids of a valid page must lie in [0, num_pages).  A page id outside that
 * range masks that page's tokens and sets the bounds bit reported by
 * fa_device_error().  Entries of pages past a sequence's length, and token
 * slots past its length in its last page, may hold anything (NaN included).
 * A contiguous cache with per-sequence lengths is the case page_size = cap,
 * max_pages = 1, page_table[b] = b.  Other rules as fa_decode_fwd.
 *
 * Scheduling: while the batch has fewer (sequence, kv head) units than SMs,
 * the kernels read the lengths on the device and give each sequence a number
 * of splits in proportion to its length (one CTA per SM), so a batch of very
 * different lengths keeps every SM streaming; otherwise each unit's share of
 * the SMs is sized from the capacity.  Either way the lengths are never read
 * on the host.
 */
int fa_decode_paged_fwd(const void* q, const void* kpages, const void* vpages,
                        const int32_t* page_table, const int32_t* seqlens, void* o, float* lse,
                        int B, int Sq, int Hq, int Hkv, int num_pages, int page_size,
                        int max_pages, int D, float scale, cudaStream_t stream);

/*
 * fa_decode_fwd_lse -- fa_decode_fwd that also writes
 *
 *   lse    [B, Hq]  fp32, 4-byte aligned, written: the log-sum-exp of each
 *          head's scores over the L valid tokens; -inf when L == 0.
 *
 * Everything else as fa_decode_fwd; lse == NULL is FA_ERR_INVALID_ARG.
 */
int fa_decode_fwd_lse(const void* q, const void* kcache, const void* vcache,
                      const int32_t* valid_len_dev, void* o, float* lse,
                      int B, int Hq, int Hkv, int cap, int D, float scale,
                      cudaStream_t stream);

/*
 * fa_decode_fwd_noalloc -- fa_decode_fwd for callers that cannot allocate
 * device memory during the call.
 *
 * No counterpart in the source material: the pages describe no
 * allocation-free variant; this is a deployment convenience of this library.
 *
 * Same arguments, layouts, results and errors as fa_decode_fwd, but the split
 * partials live in one fixed device array inside the library (4 MiB of fp32,
 * held by every GPU that loads the library until the process exits) instead of
 * memory from cudaMallocAsync.  It calls no allocating routine.  Meant for
 * code that must not allocate while it runs: serving loops with memory reserved
 * once at start-up, code running under an allocator lock, runtimes that forbid
 * allocation after initialisation.
 *
 * - Requests whose partials need more than the array holds
 *   (B * Hq * nsplit * (D + 2) floats, nsplit <= SM count) return
 *   FA_ERR_TOO_LARGE and enqueue nothing.
 * - The array is shared by all calls on a device: calls whose kernels overlap
 *   on the GPU (different streams with no ordering) race on it; calls ordered
 *   on one stream are safe.  No contents need to start at zero.
 * - The first call on each device looks up the array's device address
 *   (cudaGetSymbolAddress, with that device current).  Make that first call
 *   before any stream capture on the device.
 */
int fa_decode_fwd_noalloc(const void* q, const void* kcache, const void* vcache,
                          const int32_t* valid_len_dev, void* o,
                          int B, int Hq, int Hkv, int cap, int D, float scale,
                          cudaStream_t stream);

/*
 * fa_backward -- gradients of the loss sum(O * dout) with respect to q, k and
 * v (the flash-attention backward of tessera #90's backward commit note:
 * a "_pre" pass Delta = rowsum(dout * O), then dQ and dK/dV passes that
 * recompute P from the forward's log-sum-exp).
 *
 *   q, o, dout [B, Sq, Hq, D]    the forward's inputs, output, and the
 *                                output gradient (dtype), read only
 *   k, v       [B, Sk, Hkv, D]   read only
 *   lse        [B, Hq, Sq] fp32  the forward's log-sum-exp
 *                                (fa_prefill_fwd_lse), read only
 *   dq         [B, Sq, Hq, D]    written
 *   dk, dv     [B, Sk, Hkv, D]   written; query heads of a GQA group add
 *                                into their kv head
 *   scale, causal                as in the forward call
 *
 * Delta lives in stream-ordered scratch (B * Hq * Sq fp32).  Three kernels
 * are enqueued.  Other rules as fa_prefill_fwd.
 */
int fa_backward(const void* q, const void* k, const void* v, const void* o,
                const void* dout, const float* lse, void* dq, void* dk, void* dv,
                int B, int Hq, int Hkv, int Sq, int Sk, int D, float scale, int causal,
                int dtype, cudaStream_t stream);

/*
 * fa_prefill_fwd_host -- fa_prefill_fwd from host memory to host memory, with
 * the copies overlapped with the kernels.
 *
 *   q_host, o_host  [B, Sq, Hq, D]   in host memory (read / written)
 *   k_host, v_host  [B, Sk, Hkv, D]  in host memory (read)
 *   n_pieces        >= 1: query-row pieces per sequence (16 suits long
 *                   sequences; 1 = copies and kernel one after the other)
 *   other arguments as fa_prefill_fwd.
 *
 * Host buffers should be page-locked (cudaHostAlloc / cudaHostRegister):
 * with pageable memory the result is the same but the copies do not overlap.
 * The query rows of each sequence are split into at most n_pieces pieces on
 * 256-row boundaries; rows [s0, s1) see the key prefix [0, sk), sk = Sk, or
 * with causal masking min(Sk, max(0, s1 + Sk - Sq)), and form an ordinary
 * bottom-right aligned prefill of s1 - s0 rows over sk keys -- the same rows
 * and keys as in the whole problem, so O is bit-identical to fa_prefill_fwd's.
 * K and V are uploaded first, then Q piece by piece (heaviest piece first);
 * each piece's kernel runs as soon as its rows have landed and its O rows go
 * back while later pieces compute.
 *
 * Device copies of q, k, v, o are allocated stream-ordered on `stream`
 * (2 * B * (Sq * Hq + Sk * Hkv) * D * 2 bytes, freed on `stream` after the
 * last download).  Two copy streams and two compute streams per device (the
 * pieces' kernels alternate between them, so each fills the SMs the other's
 * last wave leaves idle), created on first use and kept, fork from `stream`
 * and join it again: work already on
 * `stream` runs first, and `stream` waits for the last download, so o_host is
 * complete once `stream` reaches that point (the call itself does not
 * synchronise).  Calls on one device are enqueued one at a time.
 *
 * Returns FA_OK, FA_ERR_INVALID_ARG (as fa_prefill_fwd, null host pointer,
 * n_pieces < 1) or FA_ERR_CUDA.
 */
int fa_prefill_fwd_host(const void* q_host, const void* k_host, const void* v_host,
                        void* o_host, int B, int Hq, int Hkv, int Sq, int Sk, int D,
                        float scale, int causal, int dtype, int n_pieces, cudaStream_t stream);

/*
 * fa_prefill_host_pieces -- the piece plan of fa_prefill_fwd_host, for
 * inspection and tests: fills b, s0, s1, sk (each may be NULL) for the first
 * min(count, max_pieces) pieces in the order they are uploaded, and returns
 * count, or -1 on bad arguments.  No GPU access.
 */
int fa_prefill_host_pieces(int B, int Sq, int Sk, int causal, int n_pieces,
                           int* b, int* s0, int* s1, int* sk, int max_pieces);

/*
 * fa_qk_norm_rope -- RMS norm of every query and key head, then the rotation
 * by position, in one pass: what prepares q and k for fa_prefill_fwd.
 * (No counterpart in the source material: an operator next to attention that
 * models with normed heads need.)
 *
 *   q      [T, Hq, D]    bf16 or fp16; token t's heads start at q + t * q_stride
 *   k      [T, Hkv, D]   elements (so q and k may be views of one projection's
 *                        output); strides are multiples of 8, at least H * D
 *   q_out  [T, Hq, D], k_out [T, Hkv, D]   contiguous, written; may be q and k
 *          themselves where those are contiguous
 *   q_weight, k_weight   [D], the heads' dtype
 *   inv_freq   [rot_dim / 2] fp32, device: radians per position of each pair
 *   positions  [T] int32, device: any value
 *   rot_dim    a multiple of 16, at most D: the rotated elements of a head
 *   eps        > 0
 *   interleaved  nonzero: pairs (2i, 2i + 1); 0: pairs (i, i + rot_dim / 2)
 *
 *   y = x / sqrt(mean(x^2) + eps) * weight; a pair (a, b) at position p turns by
 *   p * inv_freq[i]: (a cos - b sin, b cos + a sin); elements at rot_dim and
 *   past it pass through.
 *
 * fp32 arithmetic, one rounding.  Angles are 64-bit fixed-point phases: with
 * frequencies up to 1 as good as fp32's rounding of the cosine and sine at
 * |position| < 2^28, and within 2 pi 2^-23 of a radian at 2^31.  Hq or Hkv may be 0 (that side's pointers are
 * then not used).
 */
int fa_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out,
                    const void* q_weight, const void* k_weight, const float* inv_freq,
                    const int32_t* positions, long long T, int Hq, int Hkv, int D, int rot_dim,
                    long long q_stride, long long k_stride, float eps, int interleaved,
                    int dtype, cudaStream_t stream);

/*
 * fa_qk_norm_rope_append -- the serving form: the N new tokens of each of B
 * sequences are normed and rotated, k and v written straight into the pages
 * that fa_decode_paged_fwd and fa_decode_tree_fwd read.
 *
 *   q [B, N, Hq, D], k, v [B, N, Hkv, D]   token strides in elements as above
 *   q_out            [B, N, Hq, D]         contiguous; may be q
 *   kpages, vpages   [num_pages, page_size, Hkv, D]   same dtype
 *   page_table       [B, max_pages] int32, device
 *   seqlens          [B] int32, device: valid length L including the N tokens;
 *                    token s is written to slot L - N + s
 *   positions        [B, N] int32, device, or NULL: the slot.  (Nodes of a
 *                    drafted tree sit at L - N + depth.)
 *   page_size        a positive multiple of 32
 *
 * Tokens of a sequence with L < N (padding of the batch) write no cache row;
 * neither do tokens whose length passes max_pages * page_size or whose page id
 * lies outside [0, num_pages), which sets the bounds bit of fa_device_error().
 * q_out is written for every token.  Two tokens must not share a slot.
 */
int fa_qk_norm_rope_append(const void* q, const void* k, const void* v, void* q_out,
                           void* kpages, void* vpages, const void* q_weight,
                           const void* k_weight, const float* inv_freq,
                           const int32_t* positions, const int32_t* page_table,
                           const int32_t* seqlens, int B, int N, int Hq, int Hkv, int num_pages,
                           int page_size, int max_pages, int D, int rot_dim, long long q_stride,
                           long long k_stride, long long v_stride, float eps, int interleaved,
                           int dtype, cudaStream_t stream);

/*
 * fa_qk_norm_rope_backward -- gradient of fa_qk_norm_rope.
 *
 *   dq_out [T, Hq, D], dk_out [T, Hkv, D]   gradients of the outputs, contiguous
 *   q, k, weights, inv_freq, positions ...  the forward's inputs
 *   dq, dk                 contiguous, written; may be dq_out and dk_out
 *   dq_weight, dk_weight   [D] fp32, written (summed over tokens and heads in
 *                          a fixed order, so equal calls give equal bits)
 *
 * Both weight gradients are always written: a side without rows (T == 0, or no
 * heads) gets zeros.  Block sums of the weight gradients live in stream-ordered
 * scratch.
 */
int fa_qk_norm_rope_backward(const void* dq_out, const void* dk_out, const void* q,
                             const void* k, const void* q_weight, const void* k_weight,
                             const float* inv_freq, const int32_t* positions, void* dq, void* dk,
                             float* dq_weight, float* dk_weight, long long T, int Hq, int Hkv,
                             int D, int rot_dim, long long q_stride, long long k_stride,
                             float eps, int interleaved, int dtype, cudaStream_t stream);

/*
 * fa_decode_tree_fwd -- attention of a tree of drafted tokens over a paged
 * cache: fa_decode_paged_fwd for several continuations at once (speculative
 * decoding with a tree instead of a chain).
 *
 *   q, o             [B, N, Hq, D]   bf16 or fp16; N <= 64 tree nodes
 *   kpages, vpages   [num_pages, page_size, Hkv, D]
 *   page_table       [B, max_pages] int32, device
 *   seqlens          [B] int32, device: valid length L including the N nodes;
 *                    node s's K/V are in slot L - N + s
 *   parents          [B, N] int32, device: node s's parent, a lower node, or -1
 *                    (a root: its context is the cache alone), or -2 (unused)
 *   lse              NULL, or [B, N, Hq] fp32: each row's log-sum-exp
 *   page_size        a positive multiple of 32
 *
 * Node s attends to the keys [0, L - N), to its ancestors and to itself.  A
 * chain (parents[s] = s - 1) gives fa_decode_paged_fwd's rows.
 *
 * Rows of unused nodes (and of nodes below an unused one) give O = 0 and lse
 * = -inf; so do all rows of a sequence with L < N (padding of the batch).  A
 * parent entry that is no lower node makes its node unused, a length past
 * max_pages * page_size makes its sequence padding, and a page id outside [0,
 * num_pages) masks that page's keys; each sets the bounds bit of
 * fa_device_error().  Slots of unused nodes, slots at L and past it, and pages
 * past a sequence's length may hold anything (NaN included).  The K/V of the
 * used nodes and of the keys before them must be finite, as a non-finite V
 * reaches the rows that do not see it too.
 *
 * Arithmetic as fa_prefill_fwd: fp32 but for P, which is rounded to the inputs'
 * type before P V.  A row with a score that is NaN has O and lse NaN.  The tensor
 * cores' fp32 additions truncate, so O loses about 7e-7 of its size per 128-key
 * tile that one SM adds up (1e-4 in one sequence of 3 million tokens, 0.4 % at 100
 * million); lse does not.  The K/V tiles of all sequences are cut into
 * equal shares on the device, so lengths are never read on the host; shares
 * that end inside a sequence meet in fp32 partials in stream-ordered scratch
 * and are merged in a fixed order by a second kernel.  Equal calls give equal
 * bits.  Returns FA_ERR_UNSUPPORTED for N > 64, else as fa_decode_paged_fwd.
 */
int fa_decode_tree_fwd(const void* q, const void* kpages, const void* vpages,
                       const int32_t* page_table, const int32_t* seqlens,
                       const int32_t* parents, void* o, float* lse, int B, int N, int Hq,
                       int Hkv, int num_pages, int page_size, int max_pages, int D, float scale,
                       int dtype, cudaStream_t stream);

/*
 * fa_verify_tree -- which path of a drafted tree the target accepts, and the
 * token after it, from given random numbers.
 *
 *   target_probs  [B, N, V] fp32: the target's distribution after each node
 *   draft_probs   [B, N, V] fp32: the distribution from which the children of
 *                 each node were drawn (independently); or NULL: the drafts
 *                 were chosen outright (greedily, or by top-k)
 *   tokens        [B, N] int32: each node's token (node 0's is not looked at)
 *   parents       [B, N] int32: as in fa_decode_tree_fwd; node 0 is the root
 *                 (the last decided token) whatever its entry says, further
 *                 nodes with -1 or -2 are never reached
 *   uniforms      [B, N] fp32 in [0, 1): entry s >= 1 decides on node s, entry
 *                 0 draws the next token
 *   path          [B, N] int32, written: the accepted nodes, root first, then -1
 *   count         [B] int32, written: how many (at least 1, the root)
 *   next_token    [B] int32, written: the token drawn after the path's last node
 *
 * At a node with residual r = target_probs and mass Z = 1 the children are
 * tried in index order.  Child c with token x is accepted if u_c q(x) Z < r(x);
 * the walk goes on from it.  Else r becomes max(r - Z q, 0) and Z its sum; with
 * draft_probs NULL, q(x) counts as 1, r(x) becomes 0 and Z becomes Z - r(x).
 * When no child is left, the next token is the lowest whose cumulative r
 * exceeds u_0 times the sum of r.  A residual without mass falls back to the
 * node's target row; without mass there, the token is -1.  Probabilities that
 * are not positive finite numbers count as 0.
 *
 * Tests, residuals and sums are carried to at least 46 bits of the node's rows:
 * the answers are those of 64-bit arithmetic except where u lies within about
 * 2^-46 C / Z of a border, Z the mass that is left at the node and C one more than
 * the masses before it.  (1e-13 at a node's first children; 1e-11 where a draft
 * close to the target, rejected, leaves a mass of a thousandth.)  N <= 64 (else FA_ERR_UNSUPPORTED), 1 <= V < 2^30.  A token
 * outside [0, V) or a parent that is no lower node (nor -1, -2) makes its node
 * unreachable and sets the bounds bit of fa_device_error().
 */
int fa_verify_tree(const float* target_probs, const float* draft_probs, const int32_t* tokens,
                   const int32_t* parents, const float* uniforms, int32_t* path,
                   int32_t* count, int32_t* next_token, int B, int N, int V,
                   cudaStream_t stream);

/*
 * fa_compact_tree -- keeps the accepted path of a drafted tree in the cache:
 * node path[b][i] of sequence b (slot L - N + path[b][i]) moves to slot
 * L - N + i, for i < count[b], in K and V of every layer, in place; the
 * sequence's length becomes L - N + count[b].
 *
 *   kpages, vpages  [layers, num_pages, page_size, Hkv, D], 16-bit elements
 *   page_table      [B, max_pages] int32, device
 *   seqlens         [B] int32, device: lengths L including the N nodes
 *   path            [B, N] int32, device: rising node numbers (fa_verify_tree's)
 *   count           [B] int32, device: in [0, N]
 *   seqlens_out     [B] int32, device, written; may be seqlens
 *   N <= 64 (else FA_ERR_UNSUPPORTED); page_size a positive multiple of 32;
 *   layers and B at most 65535
 *
 * A sequence with L < N (padding) keeps its rows and its length.  So does one
 * whose length, count, path or page ids are out of range or whose path does
 * not rise; that sets the bounds bit of fa_device_error().  Slots behind the new
 * length keep what they held.  The pages under a sequence's tree must not be
 * shared with another sequence.
 */
int fa_compact_tree(void* kpages, void* vpages, const int32_t* page_table,
                    const int32_t* seqlens, const int32_t* path, const int32_t* count,
                    int32_t* seqlens_out, int layers, int B, int N, int Hkv, int num_pages,
                    int page_size, int max_pages, int D, cudaStream_t stream);

/* Static, human-readable name of a status code (never NULL). */
const char* fa_status_string(int status);

/*
 * fa_device_error -- read (and if reset != 0, clear) the device-side error
 * words of the current device.  Synchronises the current device.  Returns
 * FA_OK if no kernel reported a failure, FA_ERR_TIMEOUT if a pipeline wait
 * hit its time limit, FA_ERR_BOUNDS if only bounds checks fired (packed
 * offsets or page ids out of range, or an index self-check), FA_ERR_CUDA if
 * the read itself failed.
 * If detail != NULL it receives the raw bits: the prefill (and backward) word
 * in bits 0-15, the decode word (also of the cache append, tree decode,
 * verification and compaction) in bits 16-31; in each, bit 0 = a wait timed out (bits 8-15:
 * which wait), bit 1 = a bounds check fired.  Bounds bit with site 15: the
 * D = 128 backward dK/dV kernel found its dynamic shared memory too far from
 * a 1 KiB boundary to lay out its rings, and its CTAs left without work.
 */
int fa_device_error(int reset, unsigned int* detail);

/*
 * fa_last_cuda_error -- the raw cudaError_t behind the most recent
 * FA_ERR_CUDA returned to the calling thread (0 if none), and, if site is not
 * NULL, a static string naming the call that failed.
 */
int fa_last_cuda_error(const char** site);

/* Number of SMs the persistent prefill grid uses on the current device
 * (queried once per device), or a negative value on failure. */
int fa_num_sms(void);

/*
 * fa_prefill_rescale_count -- how often the prefill softmax took its lazy
 * rescale on the current device since the last reset: the number of
 * (query row, K/V tile) steps at which O and the row sum were rescaled to a
 * new running max and the tile's P recomputed.
 *
 * The lazy rescale is the "lazy" lever of "Dense flash-attention prefill
 * (gfx950 / MI355X)", *Measured*: the softmax exponentiates each K/V tile
 * against the row's running max without first taking the tile's own max, and
 * only when the tile's row sum of P exceeds 2^60 (bf16 P) or 2^15 (fp16 P),
 * or the row had no finite score before, does it find the new max, rescale
 * and recompute.  Scores of ordinary inputs never trigger it; a count that
 * grows on a workload says its scores jump by tens of units within rows.
 *
 *   reset  nonzero: clear the counter after reading it
 *   count  receives the value (non-NULL)
 *
 * Synchronises the current device.  Returns FA_OK, FA_ERR_INVALID_ARG
 * (count == NULL) or FA_ERR_CUDA.
 */
int fa_prefill_rescale_count(int reset, unsigned long long* count);

/*
 * fa_set_wait_limit_ns -- time limit of every device-side pipeline wait
 * (mbarrier waits of the prefill, decode, backward, norm and rotation and tree
 * decode kernels) on the current device; ns == 0 restores the default of 2 s.
 *
 * A wait that runs past the limit makes its CTA abort: every warp leaves its
 * loop, the loads and MMAs already in flight are waited for (each such
 * teardown wait keeps the fixed 2 s limit), tensor memory is freed, and the
 * timeout bit plus the wait's site are set in the error word read by
 * fa_device_error().  The outputs of an aborted call are undefined.  The
 * default is far above any wait of a healthy call; a short limit serves as a
 * watchdog, or in tests to make the timeout path run.
 *
 * Below 1 ms the limit is a watchdog: the decode kernels, the norm and rotation,
 * the tree decode's loads, and the dense
 * prefill (whose launches then use a polling instantiation of the kernel),
 * check it at every probe of every wait.  The packed-sequence prefill and the
 * backward kernels keep suspending probes of about 4 us each, so there a wait
 * trips the watchdog only once it has lasted about two of them (so too in the
 * tree decode's arithmetic).
 *
 * Synchronises the current device and applies to calls enqueued afterwards.
 * Returns FA_OK or FA_ERR_CUDA.
 */
int fa_set_wait_limit_ns(unsigned long long ns);

/*
 * fa_release_scratch -- gives the scratch memory that is kept for later calls on
 * the current device back to the driver.
 *
 * The tree decode and the norm and rotation's gradient take their stream-ordered
 * scratch from a memory pool of this library's, outside any framework's
 * allocator, which keeps up to 256 MiB per device of what calls have freed (the
 * device's default pool would give it back at every synchronisation, and the
 * next call would wait for the driver).  Memory that calls in flight still use is
 * kept; captured graphs own theirs.  Does not wait for the GPU.
 * Returns FA_OK or FA_ERR_CUDA.
 */
int fa_release_scratch(void);

/*
 * fa_prefill_work_item -- host copy of the persistent scheduler's work-item
 * decode, for inspection and tests.  Work item w in [0, n_items) maps to
 * (b, hq, qblock); a qblock is 256 query rows.  Returns the number of items
 * n_items = B * Hq * ceil(Sq / 256), and fills *b, *hq, *qblock when
 * 0 <= w < n_items (the pointers may be NULL).  Returns -1 on bad arguments.
 *
 * Items are numbered kv-head-major, longest causal query blocks first.  In a
 * dense launch the persistent CTAs claim items in that order from a work
 * counter (the next free CTA takes the next item).  (Packed sequences,
 * fa_prefill_varlen_fwd, claim from a list planned on the device instead.)
 */
int fa_prefill_work_item(int w, int B, int Hq, int Hkv, int Sq, int Sk, int causal,
                         int* b, int* hq, int* qblock);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_H */
