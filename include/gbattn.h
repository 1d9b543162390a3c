/*
 * gbattn.h — C ABI of the fused exact-attention library (libgbattn.so).
 *
 * The library computes exact scaled-dot-product attention
 *
 *     O = dropout(softmax(scale * Q K^T + mask)) V
 *
 * on one GPU (sm_103a) as a single tiled kernel that never writes the N x N
 * score or probability matrix to device memory, and the matching backward
 * pass that recomputes the probabilities tile by tile from Q, K and the
 * stored log-sum-exp.  The operation is the attention chain of
 * anthology-of-the-sota practice SOTA-114 ("The general form of the practice
 * above it": matmul, scale, mask, softmax, dropout, matmul fused into one
 * kernel) computed with the online-softmax tiling of "Why FlashAttention Is a
 * Kernel Story" (section "Tiling: fitting the work inside SRAM"); the
 * backward's recomputation is the one that page describes under "When it falls
 * down" (backward-pass complexity).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  Layout     Q, O, dO, dQ are contiguous [B, H, N, d] arrays and K, V, dK,
 *             dV contiguous [B, H, Nk, d] arrays, d innermost (row-major), one
 *             element type for all of them (O is bf16 for e4m3 inputs).  N is the number of query rows and
 *             Nk the number of keys (Nk = N for self-attention).  LSE is a
 *             contiguous float [B, H, N] array.  key_lens is an int32 [B]
 *             array.  Every pointer is a DEVICE pointer.
 *  Alignment  Every tensor pointer must be 16-byte aligned
 *             (ATTN_ERR_MISALIGNED otherwise).
 *  Types      ATTN_DTYPE_BF16: bf16 storage, bf16 x bf16 products with fp32
 *             accumulation.  ATTN_DTYPE_FP16: the same with IEEE half
 *             storage and f16 x f16 products (P and dS are rounded to f16).
 *             ATTN_DTYPE_FP32: fp32 storage, TF32 products with fp32
 *             accumulation (forward only, d = 64).
 *             ATTN_DTYPE_FP8_E4M3: Q, K, V stored as e4m3 (OCP FP8, one byte,
 *             no infinities), e4m3 x e4m3 products with fp32 accumulation; P
 *             is rounded to e4m3 (nearest even) for the P V product while l
 *             and LSE use the unrounded P; O is written as bf16.  Forward
 *             only, d = 128.  Per-tensor scales of quantised inputs are the
 *             caller's: fold s_q * s_k into `scale` and multiply O by s_v.
 *  Shapes     d in {64, 128} (and 256 for the bf16 and fp16 forward);
 *             B, H, N, Nk >= 1; B*H*N*d and B*H*Nk*d
 *             < 2^31 elements per tensor.  Anything else returns ATTN_ERR_UNSUPPORTED or
 *             ATTN_ERR_INVALID_ARG: the library never falls back to another
 *             implementation.
 *  Mask       query i stands at key position p = i + Nk - N: with N != Nk the
 *             queries are the last N positions of the key sequence (p = i
 *             for self-attention).  Key j of sequence b is attended by query i
 *             iff j < key_lens[b] (all Nk keys when key_lens is NULL), when
 *             causal != 0, j <= p, and, when window > 0 (sliding-window
 *             attention), p - j < window and, unless causal, j - p < window;
 *             window <= 0 means no window.  Key blocks outside the mask are
 *             skipped, not computed and masked.  A query row with no valid key
 *             gets O = 0 and LSE = -inf (and zero gradients).  key_lens values
 *             outside [0, Nk] are clamped on the device and reported as
 *             ATTN_ERR_INVALID_ARG through dev_status.
 *  Scale      scale must be finite and > 0 (1/sqrt(d) is the usual choice).
 *  Dropout    0 <= dropout_p < 1.  Kept probabilities are multiplied by
 *             1/(1 - dropout_p); the softmax denominator and LSE use the
 *             undropped probabilities.  The keep bit of score (i, j) of head
 *             (b, h) comes from one 16-bit draw of Philox4x32-10 (Salmon et
 *             al., SC'11) at counter (i, j>>3, h, b) under key (lo32(seed),
 *             hi32(seed)): output word (j>>1)&3, its low half for even j and
 *             its high half for odd j.  The score is dropped iff that draw <
 *             floor(dropout_p * 2^16), so dropout_p acts rounded down to a
 *             multiple of 2^-16.
 *             attn_bwd must get the same dropout_p, seed, causal and key_lens
 *             as the attn_fwd whose O and LSE it is given.
 *  Ownership  The caller owns every buffer, including the workspace.  The
 *             library never allocates, frees or synchronises.
 *  Streams    stream is a cudaStream_t (NULL = the legacy default stream).
 *             Work is enqueued asynchronously; outputs are valid once the
 *             stream has reached the work.  Kernels are launched with
 *             programmatic stream serialization: a kernel's blocks may be
 *             resident before the work ahead of it in the stream has
 *             finished, but no kernel touches a buffer before every earlier
 *             piece of work that may use it has finished (griddepcontrol
 *             .wait).  Inside attn_bwd the main stage loads its inputs
 *             while the preprocess runs; called by itself it starts behind all
 *             work ahead of it.
 *  Errors     Argument errors are returned before anything is enqueued, with
 *             the outputs untouched.  A failed launch returns ATTN_ERR_CUDA.
 *             Errors detected on the device (a bounded wait that expired, an
 *             out-of-range key length) are written to *dev_status (a device
 *             int, 0 = OK) when dev_status is not NULL; the kernel then exits
 *             cleanly and leaves the affected outputs unspecified.
 *  Tuning     The forward runs two 128-row query tiles per CTA (one CTA per
 *             SM) or, for bf16 and fp16 with d <= 128, one tile per CTA (two
 *             CTAs per SM): one tile by default for d = 64 with N <= 2048,
 *             else two; the environment variable GBATTN_FWD_TILES ("1" or
 *             "2", read at each call) overrides the choice.  The result does
 *             not depend on it.
 *  Threads    Every entry point is thread-safe.
 *  Devices    One process may drive several GPUs: every call runs on the
 *             device current in the calling thread (cudaSetDevice), whose
 *             context gets its own one-time kernel set-up on first use, and
 *             all pointers of a call must be memory of that device.  The library must not outlive a reset of
 *             a device it has used (cudaDeviceReset): what it set up in the
 *             old context is not redone in the new one.
 */
#ifndef GBATTN_H
#define GBATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ATTN_OK = 0,
    ATTN_ERR_INVALID_ARG = 1,    /* NULL pointer, bad size, scale, dropout_p or key length */
    ATTN_ERR_UNSUPPORTED = 2,    /* d, dtype or pass not built (never a silent fallback) */
    ATTN_ERR_MISALIGNED = 3,     /* a tensor pointer is not 16-byte aligned */
    ATTN_ERR_WORKSPACE = 4,      /* workspace NULL or smaller than attn_bwd_workspace_size */
    ATTN_ERR_CUDA = 5,           /* a CUDA runtime or driver call failed */
    ATTN_ERR_DEVICE_TIMEOUT = 6  /* (dev_status only) a bounded device-side wait expired */
} attn_status;

typedef enum {
    ATTN_DTYPE_BF16 = 0,
    ATTN_DTYPE_FP32 = 1,
    ATTN_DTYPE_FP16 = 2,
    ATTN_DTYPE_FP8_E4M3 = 3
} attn_dtype;

/*
 * Forward pass.
 *   Q         in   [B, H, N, d]
 *   K, V      in   [B, H, Nk, d]
 *   O         out  [B, H, N, d]  (same dtype as Q; bf16 for e4m3 Q, K, V)
 *   LSE       out  [B, H, N] float: natural log of the sum over valid keys of
 *                  exp(scale * q_i . k_j) (-inf for a row with no valid key)
 * One kernel launch.  Supported: bf16 and fp16 with d in {64, 128, 256}; fp32
 * (TF32 products) with d = 64; e4m3 with d = 128.
 */
attn_status attn_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE,
                     int B, int H, int N, int Nk, int d, attn_dtype dtype, float scale,
                     int causal, int window, const int32_t* key_lens, float dropout_p,
                     uint64_t seed, int* dev_status, void* stream);

/*
 * Bytes of device workspace attn_bwd needs: per head, the row terms
 * D_i = dO_i . O_i and the log-sum-exp in base 2 (two floats per row) and an
 * fp32 accumulator for dQ, with N (query rows) rounded up to a multiple of
 * 128.  It does not depend on Nk.  Returns 0 for arguments attn_bwd would
 * reject.
 */
size_t attn_bwd_workspace_size(int B, int H, int N, int d);

/*
 * Backward pass: given the forward's inputs, its O and LSE and the incoming
 * gradient dO, writes dQ ([B, H, N, d]) and dK, dV ([B, H, Nk, d]), in the
 * dtype of Q.  bf16 or fp16, d in {64, 128}.  workspace must hold
 * attn_bwd_workspace_size(B, H, N, d) bytes (16-byte aligned); its contents
 * on entry do not matter.  Enqueues
 * three launches: attn_bwd_preprocess, attn_bwd_main, attn_bwd_dq_convert.
 */
attn_status attn_bwd(const void* Q, const void* K, const void* V, const void* O,
                     const void* dO, const float* LSE, void* dQ, void* dK, void* dV,
                     int B, int H, int N, int Nk, int d, attn_dtype dtype, float scale,
                     int causal, int window, const int32_t* key_lens, float dropout_p,
                     uint64_t seed, void* workspace, size_t workspace_bytes, int* dev_status,
                     void* stream);

/*
 * The three stages of attn_bwd, exported so that a caller can enqueue (and
 * time) them one by one.  Same arguments and rules as attn_bwd; calling the
 * three in this order on one stream with one workspace is exactly attn_bwd.
 *   preprocess: D_i = dO_i . O_i and -LSE_i * log2(e) into the workspace;
 *               clears the dQ accumulator.
 *   main:       recomputes P tile by tile; writes dK, dV; accumulates dQ
 *               (unscaled) into the workspace.
 *   dq_convert: dQ = scale * accumulator, rounded to the output dtype.
 */
attn_status attn_bwd_preprocess(const void* O, const void* dO, const float* LSE,
                                int B, int H, int N, int d, attn_dtype dtype,
                                void* workspace, size_t workspace_bytes, void* stream);
attn_status attn_bwd_main(const void* Q, const void* K, const void* V, const void* dO,
                          void* dK, void* dV, int B, int H, int N, int Nk, int d,
                          attn_dtype dtype, float scale, int causal, int window,
                          const int32_t* key_lens, float dropout_p, uint64_t seed,
                          void* workspace, size_t workspace_bytes, int* dev_status, void* stream);
attn_status attn_bwd_dq_convert(void* dQ, int B, int H, int N, int d, attn_dtype dtype,
                                float scale, const void* workspace, size_t workspace_bytes,
                                void* stream);

/*
 * attn_bwd without a workspace argument, for callers that cannot allocate
 * device memory where they run the backward (a plugin inside a framework that
 * owns every device allocation and gives it no allocator, or latency-critical
 * code that must not call cudaMalloc).  The pages have no counterpart: this is
 * a deployment convenience, not part of the method.
 *   Scratch   a 32 MiB buffer inside the library (a file-scope __device__
 *             array), held by every GPU that loads the library until exit.
 *             Shapes whose attn_bwd_workspace_size exceeds 32 MiB are
 *             rejected with ATTN_ERR_WORKSPACE before anything is enqueued.
 *   Set-up    the first call on a device looks up the buffer's device address
 *             (cudaGetSymbolAddress) with that device current; make that first
 *             call before any stream capture.  The address is looked up again
 *             if the device's context has changed since (a device reset).
 *   Sharing   every call uses the same buffer; each call clears what must
 *             start at zero, but calls that overlap on the GPU race on it.
 *   Allocates nothing: no cudaMalloc, cudaFree or allocating library call.
 * Otherwise identical to attn_bwd (same arguments minus the workspace, same
 * results, same errors).  attn_bwd's argument errors are checked first; a
 * shape that passes them but needs more scratch than 32 MiB then returns
 * ATTN_ERR_WORKSPACE.
 */
attn_status attn_bwd_noalloc(const void* Q, const void* K, const void* V, const void* O,
                             const void* dO, const float* LSE, void* dQ, void* dK, void* dV,
                             int B, int H, int N, int Nk, int d, attn_dtype dtype, float scale,
                             int causal, int window, const int32_t* key_lens, float dropout_p,
                             uint64_t seed, int* dev_status, void* stream);

/*
 * Packed variable-length sequences (the layout of batches without padding):
 * the B sequences of a batch are concatenated along the token axis.
 *   Q, O, dO, dQ   [total_q, H, d]     K, V, dK, dV   [total_k, H, d]
 *   LSE            float [H, total_q]
 *   cu_seqlens_q   int32 [B + 1], DEVICE, 4-byte aligned: sequence b holds
 *                  query tokens [cu_seqlens_q[b], cu_seqlens_q[b+1]);
 *                  cu_seqlens_q[0] = 0 and cu_seqlens_q[B] = total_q.
 *   cu_seqlens_k   the same for the keys (may equal cu_seqlens_q).
 *   max_seqlen_q   an upper bound on every query length (sets the grid and
 *                  the workspace); max_seqlen_k the same for the keys.
 * Each sequence is attended on its own, with the mask of the dense entry
 * points applied to its lengths N_b = cu_q[b+1] - cu_q[b] and
 * Nk_b = cu_k[b+1] - cu_k[b] (queries are the last N_b key positions; no
 * key_lens).  The dropout counter is (i, j>>3, h, b) with i, j counted within
 * sequence b.  bf16 or fp16 only.  Offsets that leave [0, total], decrease,
 * or give a sequence longer than its max_seqlen are clamped on the device
 * (no access leaves the tensors) and reported as ATTN_ERR_INVALID_ARG through
 * dev_status.  attn_bwd_varlen's workspace holds
 * attn_bwd_workspace_size(B, H, max_seqlen_q, d) bytes.  Otherwise the
 * conventions above hold; one launch for the forward, three for the backward.
 */
attn_status attn_fwd_varlen(const void* Q, const void* K, const void* V, void* O, float* LSE,
                            const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                            int B, int H, int total_q, int total_k, int max_seqlen_q,
                            int max_seqlen_k, int d, attn_dtype dtype, float scale, int causal,
                            int window, float dropout_p, uint64_t seed, int* dev_status,
                            void* stream);
attn_status attn_bwd_varlen(const void* Q, const void* K, const void* V, const void* O,
                            const void* dO, const float* LSE, void* dQ, void* dK, void* dV,
                            const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                            int B, int H, int total_q, int total_k, int max_seqlen_q,
                            int max_seqlen_k, int d, attn_dtype dtype, float scale, int causal,
                            int window, float dropout_p, uint64_t seed, void* workspace,
                            size_t workspace_bytes, int* dev_status, void* stream);

/*
 * Serving from a paged key/value cache.  A decoding server keeps the keys and
 * values of its requests in pages of a common pool, because their lengths
 * grow and cannot be known ahead.  One step runs three entry points:
 * attn_page_table gives the step's new tokens their slots, attn_cache_append
 * writes their K and V rows there, attn_fwd_paged attends over the cache.
 *   cache      k_cache, v_cache: [num_pages, H_kv, page_size, d], bf16 or fp16,
 *              the same strides for both, d innermost.  The strides of page,
 *              head and token (in elements, multiples of 8) are arguments, so
 *              a cache may be a view: token-major pages [num_pages, page_size,
 *              H_kv, d], or K and V side by side in one array.  The stride of
 *              a dimension of extent 1 is ignored.  page_size is a multiple of
 *              8; num_pages * page_size < 2^31.
 *   page_table int32 [B, max_pages], contiguous: entry [b, c] is the page that
 *              holds keys [c page_size, (c+1) page_size) of request b.  Entries
 *              past a request's last key, or before every key that its window
 *              still reaches, are not used.  max_pages * page_size <= 2^30.
 *   slot       page * page_size + row: the place of one token in the pool.
 *   lengths    int32 device arrays, so that a step captured into a graph can
 *              be replayed with other lengths.
 * No backward pass: the cache serves inference.  Conventions (streams, errors,
 * alignment, ownership) as above.
 */

/*
 * Page table and slot map of one step.  Request b has cached_lens[b] tokens in
 * the cache and gets new_lens[b] more (either may be 0).
 *   cu_seqlens_q  out [B + 1]  exclusive sums of new_lens
 *   seq_lens      out [B]      cached_lens + new_lens
 *   page_table    in/out       the pages that request b holds, entries [0,
 *                              ceil(cached_lens[b] / page_size)), are read; the
 *                              pages its new tokens need beyond them are
 *                              entered behind; nothing else is written.  Requests
 *                              that get new tokens may share full pages, not the
 *                              one that their cached tokens end in
 *   slots         out int64 [max_tokens]  slot of each packed new token; -1
 *                              from the last token on
 *   pages_taken   out [1]      free pages used
 *   free_pages    in [free_capacity], num_free in [1]: a stack of page ids,
 *                              free_pages[0, num_free).  Pages are taken from
 *                              its end, request by request: the i-th taken is
 *                              free_pages[num_free - 1 - i].  The caller lowers
 *                              num_free by pages_taken.
 * Outputs must not overlap inputs or one another (ATTN_ERR_INVALID_ARG), page_table
 * apart, which is both.  B, max_pages, max_tokens, free_capacity >= 1.  Clamped and reported
 * as ATTN_ERR_INVALID_ARG through dev_status: negative lengths (to 0),
 * requests longer than max_pages pages (their new tokens are cut), new tokens
 * past max_tokens (cut), num_free outside [0, free_capacity].  When the free
 * pages run out, the pages missing are entered as -1 and their tokens' slots
 * are -1 (reported too).  B <= 16384, max_tokens <= 2^30.  One launch.
 */
attn_status attn_page_table(const int32_t* cached_lens, const int32_t* new_lens,
                            int32_t* page_table, const int32_t* free_pages,
                            const int32_t* num_free, int32_t* cu_seqlens_q, int32_t* seq_lens,
                            int64_t* slots, int32_t* pages_taken, int B, int max_pages,
                            int page_size, int max_tokens, int free_capacity, int* dev_status,
                            void* stream);

/*
 * Writes row t of K and V ([T, H_kv, d], d innermost, the given token and head
 * strides for both) to slot slots[t] of every head of the caches.  A slot of
 * -1 is skipped; any other slot outside [0, num_pages * page_size) is skipped
 * and reported as ATTN_ERR_INVALID_ARG through dev_status.  Slots must differ
 * from one another: what a slot named twice holds is unspecified.  K and V
 * must not overlap the caches.  T >= 1; bf16 or fp16, d in {64, 128, 256}.  One launch.
 */
attn_status attn_cache_append(const void* K, const void* V, void* k_cache, void* v_cache,
                              const int64_t* slots, int T, int H_kv, int d, attn_dtype dtype,
                              int64_t token_stride, int64_t head_stride, int num_pages,
                              int page_size, int64_t cache_page_stride, int64_t cache_head_stride,
                              int64_t cache_token_stride, int* dev_status, void* stream);

/*
 * Attention of packed new tokens over the cache; from single tokens (decoding)
 * to whole prompts, mixed in one call.
 *   Q    in  [total_q, H, d], d innermost, the given token and head strides
 *            (multiples of 8 elements): a slice of a fused projection will do
 *   O    out [total_q, H, d] contiguous; LSE out float [H, total_q]
 *   cu_seqlens_q  int32 [B + 1]: request b's queries are rows [cu_seqlens_q[b],
 *            cu_seqlens_q[b+1]), at most max_seqlen_q of them, possibly none
 *   seq_lens int32 [B]: keys of request b, its new tokens included; possibly 0
 * Query head h reads key/value head h / (H / H_kv); H_kv divides H, at most 128
 * query heads each.  Mask, scale and LSE as in attn_fwd_varlen with Nk_b =
 * seq_lens[b]: a request's queries are its last key positions; a query without
 * a key gets O = 0 and LSE = -inf.  Cache slots that no query of a request may
 * attend (past its last key, before its window) may hold anything, NaN
 * included, without effect; a V row that some query attends is multiplied by a
 * weight of 0 for queries of the same call that do not, which keeps a NaN or an
 * infinity.  Rows of Q behind cu_seqlens_q[B] are ignored, and those of O and
 * LSE left as they are.
 * Clamped on the device (no access leaves the tensors) and reported as
 * ATTN_ERR_INVALID_ARG through dev_status: bad cu_seqlens_q as in
 * attn_fwd_varlen, seq_lens outside [0, max_pages * page_size], and page ids
 * outside [0, num_pages) (zeros are read for their keys).
 * 1 <= B, total_q <= 2^30, max_seqlen_q >= 1; bf16 or fp16, d in {64, 128, 256}.
 * Requests may share pages.  O, LSE and the workspace must not overlap the
 * inputs or one another.  The workspace holds
 * attn_fwd_paged_workspace_size(...) bytes (16-byte aligned, contents on entry
 * do not matter; may be NULL when that is 0); calls that may overlap on the
 * GPU need one each.  One to three launches.
 * Kernel and split are chosen from these sizes alone (so that a captured call
 * can be replayed with other lengths), and max_pages * page_size stands for the
 * longest context there: the result depends on it by rounding only, the time
 * can do so by much.
 */
attn_status attn_fwd_paged(const void* Q, const void* k_cache, const void* v_cache, void* O,
                           float* LSE, const int32_t* cu_seqlens_q, const int32_t* seq_lens,
                           const int32_t* page_table, int B, int H, int H_kv, int total_q,
                           int max_seqlen_q, int num_pages, int page_size, int max_pages, int d,
                           attn_dtype dtype, int64_t q_token_stride, int64_t q_head_stride,
                           int64_t cache_page_stride, int64_t cache_head_stride,
                           int64_t cache_token_stride, float scale, int causal, int window,
                           void* workspace, size_t workspace_bytes, int* dev_status,
                           void* stream);

/*
 * Bytes of device workspace attn_fwd_paged needs for partial results, where
 * the keys of a query tile are shared out over several CTAs.  0 where it needs
 * none, and for arguments that it would reject.
 */
size_t attn_fwd_paged_workspace_size(int B, int H, int H_kv, int total_q, int max_seqlen_q,
                                     int max_pages, int page_size, int d);

/*
 * Rotary positions of queries and keys.  A pair (a, b) of the first rotary_dim
 * elements of a row at position t becomes
 *     (scaling (a cos w - b sin w), scaling (b cos w + a sin w)),  w = t inv_freq[i],
 * for the pairs i = 0 .. rotary_dim / 2 - 1: elements i and i + rotary_dim / 2, or
 * with interleaved != 0 elements 2 i and 2 i + 1.  The row's other elements are
 * copied.  inverse != 0 turns by -w, with the same factor: the transposed map, which
 * gives the gradient of the inputs from that of the outputs.  Long contexts scaled by
 * interpolation, another base or by parts are other inv_freq; `scaling` is
 * the factor that some of them put on cosine and sine (else 1).
 *   Q, Q_out   [B, H, N, d], d innermost, any strides that are multiples of 16
 *              bytes: dense tensors, packed tokens [T, H, d] (B = 1, N = T), slices of
 *              a fused projection.  Strides of inputs may be 0 (a broadcast row).  The
 *              stride of a dimension of extent 1 is ignored
 *   K, K_out   [B, H_k, N, d], the same; not used when H_k = 0
 *   inv_freq   float [rotary_dim / 2], finite
 *   positions  int32, row n of batch entry b is at positions[b position_batch_stride
 *              + n] (position_batch_stride 0: the same for all b); NULL: at n.  Any
 *              value, negative ones too: an angle is off by at most
 *              |t| max(1, |inv_freq|) 2^-53 + 2^-25 turns, and cosine and sine of that
 *              angle by 2^-20 (fp32: 2^-22)
 * Q_out may be Q, and K_out K, with the same strides (in place); otherwise outputs
 * overlap neither inputs nor one another.  bf16, fp16 or fp32; d in {64, 128, 256};
 * rotary_dim a multiple of 16 up to d; N <= 2^30.  One launch.
 */
attn_status attn_rope(const void* Q, const void* K, void* Q_out, void* K_out, const float* inv_freq,
                      const int32_t* positions, int B, int H, int H_k, int N, int d, int rotary_dim,
                      attn_dtype dtype, int64_t q_batch_stride, int64_t q_head_stride,
                      int64_t q_token_stride, int64_t k_batch_stride, int64_t k_head_stride,
                      int64_t k_token_stride, int64_t q_out_batch_stride, int64_t q_out_head_stride,
                      int64_t q_out_token_stride, int64_t k_out_batch_stride,
                      int64_t k_out_head_stride, int64_t k_out_token_stride,
                      int64_t position_batch_stride, float scaling, int interleaved, int inverse,
                      void* stream);

/*
 * attn_cache_append with the rotation of attn_rope on the way: the rotated row t of
 * K and row t of V go to slot slots[t], and the rotated row t of Q to row t of
 * Q_out ([T, H, d], d innermost, the given strides; may be Q with the same strides).
 *   positions     int32 [T], or NULL:
 *   cu_seqlens_q  int32 [B + 1], seq_lens int32 [B], as attn_page_table leaves
 *                 them: token t of request b stands at seq_lens[b] -
 *                 cu_seqlens_q[b+1] + t.  Tokens behind the last request are left
 *                 out, rows of Q_out included.  (Not used where positions is given,
 *                 and all T rows of Q_out are then written.)
 * Slots as in attn_cache_append (a token without a slot still has its Q rotated);
 * a slot of a token behind the last request is reported as ATTN_ERR_INVALID_ARG.
 * T >= 1; bf16 or fp16; d and rotary_dim as in attn_rope.  One launch.
 */
attn_status attn_cache_append_rope(const void* Q, const void* K, const void* V, void* Q_out,
                                   void* k_cache, void* v_cache, const int64_t* slots,
                                   const float* inv_freq, const int32_t* positions,
                                   const int32_t* cu_seqlens_q, const int32_t* seq_lens, int B, int T,
                                   int H, int H_kv, int d, int rotary_dim, attn_dtype dtype,
                                   int64_t q_token_stride, int64_t q_head_stride,
                                   int64_t kv_token_stride, int64_t kv_head_stride,
                                   int64_t q_out_token_stride, int64_t q_out_head_stride,
                                   int num_pages, int page_size, int64_t cache_page_stride,
                                   int64_t cache_head_stride, int64_t cache_token_stride,
                                   float scaling, int interleaved, int* dev_status, void* stream);

/*
 * A paged cache held in 8 bits.  k_cache and v_cache are [num_pages, H_kv,
 * page_size, d] arrays of e4m3 with strides as above (multiples of 16 elements), and
 * k_scale and v_scale contiguous float [num_pages, H_kv] arrays: the block of a page
 * and head stands for its e4m3 values times its scale, a power of two from 2^-48 to
 * 2^48 (so that the scale adds no rounding).  The kernels go by a scale's exponent,
 * clamped to that range; one that is no power of two is reported as
 * ATTN_ERR_INVALID_ARG through dev_status.  0 counts as 2^-48 and is not reported.
 *
 * attn_cache_append_fp8 writes row t of K and V (bf16 or fp16, as in
 * attn_cache_append) to slot slots[t], rounded to the nearest e4m3 number of the block's
 * scale, ties to even.  The scale becomes the smallest one that holds all of the
 * block's rows: those that this call writes, and the rows before the first of them,
 * whose scale is the block's old one; where it grows, those rows are rounded again
 * on the new one.  A row written to a page's row 0 starts the block
 * anew: the old scale does not count.  Infinities, and values past 448 x 2^48, become
 * the largest number, and the scale 2^48, on which the block's other rows are zeros where
 * they are below 2^38; a NaN stays one and does not count for the scale.
 * The slots of a page that one call names are one ascending run of consecutive rows at
 * consecutive tokens, as attn_page_table makes them.  A slot of -1 is skipped, any other
 * slot outside the cache skipped and reported.  A second run of a page behind the first, with
 * no token between them or only tokens without a slot, as many as rows at most (a row
 * twice, out of order, or rows skipped in the middle of a page), is left out and reported as
 * ATTN_ERR_INVALID_ARG; what a page holds that is named again elsewhere in the call is
 * unspecified.  No two requests may write to one page.
 * T H_kv < 2^30.  One launch.
 */
attn_status attn_cache_append_fp8(const void* K, const void* V, void* k_cache, void* v_cache,
                                  float* k_scale, float* v_scale, const int64_t* slots, int T,
                                  int H_kv, int d, attn_dtype dtype, int64_t token_stride,
                                  int64_t head_stride, int num_pages, int page_size,
                                  int64_t cache_page_stride, int64_t cache_head_stride,
                                  int64_t cache_token_stride, int* dev_status, void* stream);

/*
 * attn_fwd_paged over a cache held in 8 bits: Q and O in bf16 or fp16 (dtype is
 * theirs), everything else as there, the workspace's size included.  Scales are read
 * for the pages with a key that some query attends.  They may be as far apart as they
 * like, a row's accuracy is that of the pages it attends; where scales within 128 keys are
 * more than 2^3 apart, chunks and prompts take up to 1.6 times as long.
 */
attn_status attn_fwd_paged_fp8(const void* Q, const void* k_cache, const void* v_cache,
                               const float* k_scale, const float* v_scale, void* O, float* LSE,
                               const int32_t* cu_seqlens_q, const int32_t* seq_lens,
                               const int32_t* page_table, int B, int H, int H_kv, int total_q,
                               int max_seqlen_q, int num_pages, int page_size, int max_pages,
                               int d, attn_dtype dtype, int64_t q_token_stride,
                               int64_t q_head_stride, int64_t cache_page_stride,
                               int64_t cache_head_stride, int64_t cache_token_stride, float scale,
                               int causal, int window, void* workspace, size_t workspace_bytes,
                               int* dev_status, void* stream);

/*
 * Device self-test of the failure detection the kernels rely on: one warp
 * waits on an mbarrier with the same bounded wait (about 2 s of
 * %globaltimer) that every kernel uses.  arrive != 0: one thread arrives
 * first, the wait succeeds and *dev_status is left as it is.  arrive == 0:
 * nothing arrives, the wait expires and ATTN_ERR_DEVICE_TIMEOUT is written to
 * *dev_status (a device int, 0 on entry).  Nothing else is in flight, so the
 * expiry leaves the context usable.  Not part of the attention path.
 */
attn_status attn_selftest_wait(int* dev_status, int arrive, void* stream);

/*
 * Device self-test of the fused forward kernel's own abort path.  It runs the
 * bf16, d = 128, non-causal forward (the kernel of attn_fwd, in a test
 * instantiation that only this entry point launches) on Q [B, H, N, 128] and
 * K, V [B, H, Nk, 128], with two changes: the producer never issues the copy
 * of the K tile of key block withhold_block (a tile withheld, not a fault:
 * nothing ever completes that tile's barrier), and every wait gives up after
 * wait_ms milliseconds (1 to 2000) instead of about 2 s.  A CTA that walks
 * that key block then has copies and MMAs in flight when its wait expires: it
 * drains them, frees its tensor memory, writes ATTN_ERR_DEVICE_TIMEOUT to
 * *dev_status (required, a device int, 0 on entry) and returns; O and LSE of
 * such CTAs are unspecified.  withhold_block < 0 withholds nothing and gives
 * the ordinary result.  Not part of the attention path.
 */
attn_status attn_selftest_fwd_withheld(const void* Q, const void* K, const void* V, void* O,
                                       float* LSE, int B, int H, int N, int Nk,
                                       int withhold_block, int wait_ms, int* dev_status,
                                       void* stream);

/* Static, NUL-terminated description of a status code. */
const char* attn_status_string(attn_status status);

/* Library version: major * 10000 + minor * 100 + patch. */
int attn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GBATTN_H */
