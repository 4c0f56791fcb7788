/*
 * gqa_attn.h -- C ABI of libgqa_attn.so: fused multi-head attention forward
 * with grouped-query attention (GQA) and split-KV single-token decode, written
 * for NVIDIA B200 (sm_100a).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Tensors are caller-owned DEVICE buffers (allocated by the caller, e.g.
 *    with PyTorch), dense and row-major (C order).  Q, K, V and O hold bf16
 *    values (raw 16-bit storage); LSE holds float32; lengths hold int32.
 *    Every tensor base address must be 16-byte aligned.
 *  - `stream` is a cudaStream_t passed as void* (NULL = the legacy default
 *    stream).  Calls are asynchronous: they validate their arguments on the
 *    host, enqueue kernels on `stream` and return.  The library never
 *    synchronises a stream except in attn_last_device_status().
 *  - Errors detectable on the host are returned before anything is enqueued:
 *    ATTN_ERR_NULL for a NULL required pointer, ATTN_ERR_INVALID for
 *    inconsistent sizes or flags, ATTN_ERR_UNSUPPORTED for a head size the
 *    library was not built for, ATTN_ERR_CUDA when a CUDA call fails.
 *  - Errors found on the device (a bounded wait that ran out, a length
 *    outside the tensor) are recorded in a per-device status word and read
 *    back with attn_last_device_status().  Kernels never trap.
 *  - Query head h reads key/value head h / (Hq / Hkv): consecutive groups of
 *    Hq / Hkv query heads share one K/V head (GQA; Heads must be a multiple of
 *    Heads_KV -- Tylo.jl "Primitives" page, entry `flex_attention!`).
 */
#ifndef GQA_ATTN_H
#define GQA_ATTN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ATTN_OK = 0,
    ATTN_ERR_NULL = 1,          /* a required pointer is NULL */
    ATTN_ERR_INVALID = 2,       /* sizes / flags inconsistent, misaligned pointer */
    ATTN_ERR_UNSUPPORTED = 3,   /* head size D not built (built: 64, 128) */
    ATTN_ERR_CUDA = 4,          /* a CUDA runtime / driver call failed */
    ATTN_ERR_TIMEOUT = 5,       /* device: a bounded wait ran out, kernel gave up */
    ATTN_ERR_DEVICE_BOUNDS = 6, /* device: a length exceeded the tensor, clamped */
    ATTN_ERR_SCRATCH_LIMIT = 7, /* attn_decode_noalloc: workspace above its fixed array */
    ATTN_ERR_NO_PAGES = 8       /* device: no free page left in the cache's pool */
} attn_status_t;

/*
 * attn_fwd -- fused attention forward, O = softmax(Q K^T * scale + mask) V.
 *
 * Defined by: Tylo.jl "Primitives" page, entry `attention!` (fused MHA with
 * GQA; keywords causal, input_pos = absolute position of the first query,
 * k_lengths / q_lengths = optional per-batch valid lengths; the softmax
 * statistics M/L are saved for the backward; Float32 accumulation), the
 * causal rule of entry `CausalMask` (a query sees keys at or before its own
 * absolute position), and the sliding window of the mlx-arsenal "Attention"
 * page, entry `sliding_window_mask` (at most window_size keys, the query's
 * own position included).
 *
 *   O     [out] bf16 (B, Hq, Sq, D)
 *   Q     [in]  bf16 (B, Hq, Sq, D)
 *   K, V  [in]  bf16 (B, Hkv, Sk, D)
 *   LSE   [out] float32 (B, Hq, Sq) or NULL (statistics not saved).
 *         LSE = M + ln L in natural-log units of the scaled scores, where
 *         M = max_j s_j and L = sum_j exp(s_j - M) over the visible keys.
 *   scale       multiplies Q K^T (the pages' default is 1/sqrt(D)).
 *   causal      0 or 1.  Key j is visible from query row i only if
 *               j <= input_pos + i.
 *   window      0 = no window; w > 0 (requires causal) keeps only keys with
 *               input_pos + i - w < j <= input_pos + i.
 *   input_pos   >= 0, absolute position of query row 0.
 *   k_lengths   int32 (B,) device array or NULL (= Sk): keys j >= k_lengths[b]
 *               are invisible.  Values above Sk are clamped to Sk and flagged
 *               ATTN_ERR_DEVICE_BOUNDS; negative values count as 0.
 *   Sizes: B, Sq, Sk >= 0; Hq, Hkv >= 1, Hq % Hkv == 0; D in {64, 128}.
 *
 * A query row that sees no key (k_length 0, or every key cut by the masks)
 * gets O = 0 and LSE = -inf.  Key/value rows at positions >= k_lengths[b]
 * contribute exactly zero, whatever they hold.
 */
attn_status_t attn_fwd(void *O, const void *Q, const void *K, const void *V, float *LSE,
                       int B, int Hq, int Hkv, int Sq, int Sk, int D, float scale,
                       int causal, int window, int input_pos,
                       const int32_t *k_lengths, void *stream);

/*
 * attn_fwd_varlen -- attn_fwd plus per-batch valid query lengths.
 *
 * Same definition and arguments as attn_fwd, with q_lengths an int32 (B,)
 * device array or NULL (= Sq): query rows i >= q_lengths[b] are invalid and
 * get O = +0.0 (every bit zero) and LSE = -inf, whatever those rows of Q hold,
 * NaN and Inf included (Tylo.jl "Primitives" page, entry `attention!`, keyword
 * q_lengths).  attn_fwd(...) is attn_fwd_varlen(..., q_lengths=NULL).
 */
attn_status_t attn_fwd_varlen(void *O, const void *Q, const void *K, const void *V, float *LSE,
                              int B, int Hq, int Hkv, int Sq, int Sk, int D, float scale,
                              int causal, int window, int input_pos,
                              const int32_t *k_lengths, const int32_t *q_lengths,
                              void *stream);

/*
 * attn_fwd_flex -- flex_attention! forward with one score mod and a document
 * mask (Tylo.jl "Primitives" page, entries `flex_attention!`,
 * `SoftCapScore`, `AliBiScore`, `DocumentMask`, `BlockMask`).
 *
 * Same tensors, masks and lengths as attn_fwd_varlen; on top of them, with
 * s = scale * <q_i, k_j> the scaled score of query row i and key j:
 *   softcap       > 0: s -> softcap * tanh(s / softcap)        (SoftCapScore)
 *   alibi_slopes  float32 (Hq,) device array or NULL:
 *                 s -> s + alibi_slopes[h] * ((input_pos + i) - j)  (AliBiScore)
 *                 At most one of softcap > 0 and alibi_slopes is given.
 *   doc_q, doc_kv int32 device arrays, (Sq,) ids of the query rows and (Sk,)
 *                 ids of the keys, both NULL or both given: the pair attends
 *                 only if the ids match (DocumentMask; shared by every batch
 *                 entry and head).
 *   block_mask    uint8 device array (ceil(Sq/64), ceil(Sk/64)) or NULL, one
 *                 state per 64x64 block of (query row, key): 0 = no pair of
 *                 the block attends (skipped), 2 = every pair attends (document
 *                 ids not checked), anything else = check each pair.  Build it
 *                 with attn_block_mask_document or attn_block_mask_build (the
 *                 page's build_block_mask); it must agree with the other masks.
 *   block_mask_per_head  0: one block_mask for every batch entry and head;
 *                 1: block_mask is (B, Hq, ceil(Sq/64), ceil(Sk/64)), one matrix
 *                 per (batch, query head) -- block-sparse prefill with the
 *                 masks of attn_rbs_block_mask.
 * A call with a block_mask and nothing else to apply (causal 0, no lengths, no
 * document ids, no score mod, Sk <= 65536) runs the block-sparse kernel, which
 * steps over the kept 64-key blocks of each 128-row query tile; it computes the
 * same function.
 * Limits: Sk <= 131072.  Errors as attn_fwd, plus ATTN_ERR_INVALID for a
 * negative or non-finite softcap, softcap together with ALiBi, or only one of
 * doc_q / doc_kv, and ATTN_ERR_UNSUPPORTED for a longer Sk.
 */
attn_status_t attn_fwd_flex(void *O, const void *Q, const void *K, const void *V, float *LSE,
                            int B, int Hq, int Hkv, int Sq, int Sk, int D, float scale,
                            int causal, int window, int input_pos,
                            const int32_t *k_lengths, const int32_t *q_lengths,
                            float softcap, const float *alibi_slopes,
                            const int32_t *doc_q, const int32_t *doc_kv,
                            const uint8_t *block_mask, int block_mask_per_head, void *stream);

/*
 * attn_bwd -- backward of attn_fwd_varlen (Tylo.jl "Primitives" page, entry
 * `∇attention!`: from the output gradient, the inputs, the output and the
 * forward's saved softmax statistics, write the input gradients; overwrite).
 *
 *   dQ  [out] bf16 (B, Hq, Sq, D);  dK, dV [out] bf16 (B, Hkv, Sk, D)
 *   dO  [in]  bf16 (B, Hq, Sq, D), the output gradient
 *   Q, K, V, O [in] the forward's inputs and output
 *   LSE [in]  float32 (B, Hq, Sq) saved by the forward (LSE = M + ln L)
 *   scale, causal, window, input_pos, k_lengths, q_lengths: as in the forward
 *   (they must match it).
 * With P = exp(scale Q K^T - LSE) on the visible pairs: dV = P^T dO,
 * dS = P (dO V^T - rowsum(dO O)), dQ = scale dS K, dK = scale dS^T Q; dK / dV
 * of a KV head sum over the query heads it serves; keys never visible and
 * query rows past q_lengths get zero gradients (rows of dQ past q_lengths and
 * of dK, dV past k_lengths are +0.0).  Padding rows (Q, dO, O past q_lengths;
 * K, V past k_lengths) must hold finite values: they enter the tensor-core
 * products with weight zero, and zero times NaN or Inf is NaN.  Allocates a
 * stream-ordered workspace of B * Hq * Sq floats.  The dQ kernel runs on a
 * library-owned stream forked from `stream` and joined back to it with events,
 * so the call stays ordered on `stream` (and can be captured in a CUDA graph).
 * Errors as attn_fwd.
 */
attn_status_t attn_bwd(void *dQ, void *dK, void *dV, const void *dO, const void *Q, const void *K,
                       const void *V, const void *O, const float *LSE, int B, int Hq, int Hkv,
                       int Sq, int Sk, int D, float scale, int causal, int window, int input_pos,
                       const int32_t *k_lengths, const int32_t *q_lengths, void *stream);

/*
 * attn_fwd_sinks -- attn_fwd_varlen with a sliding window and sinks: the first `sinks`
 * keys stay visible to every query at or past them, whatever the window.
 *
 *   visible(i, j) = j <= p and (j > p - window or j < sinks),  p = input_pos + i,
 *                   and j < k_lengths[b], i < q_lengths[b]
 *
 * Arguments, outputs and errors as attn_fwd_varlen with causal = 1, except that
 * window >= 1 is required and sinks >= 0 is added.  sinks = 0 is attn_fwd_varlen with
 * that window; a window of input_pos + Sq or more is plain causal attention.  Rows of V
 * below k_lengths[b] must hold finite values, also those that no query of the call sees:
 * they may enter products with weight zero.
 */
attn_status_t attn_fwd_sinks(void *O, const void *Q, const void *K, const void *V, float *LSE,
                             int B, int Hq, int Hkv, int Sq, int Sk, int D, float scale,
                             int window, int sinks, int input_pos,
                             const int32_t *k_lengths, const int32_t *q_lengths, void *stream);

/*
 * attn_bwd_sinks -- backward of attn_fwd_sinks: attn_bwd on that mask, with the same
 * arguments, padding rules and errors (window >= 1, sinks >= 0, as in the forward).  Its
 * workspace is attn_bwd's, plus fp32 partials where the items of a key tile are split over
 * CTAs (up to about 40 MB).
 */
attn_status_t attn_bwd_sinks(void *dQ, void *dK, void *dV, const void *dO, const void *Q,
                             const void *K, const void *V, const void *O, const float *LSE,
                             int B, int Hq, int Hkv, int Sq, int Sk, int D, float scale,
                             int window, int sinks, int input_pos,
                             const int32_t *k_lengths, const int32_t *q_lengths, void *stream);

/*
 * attn_rbs_block_mask -- block scores and block mask of block-sparse prefill
 * (mlx-arsenal "Radius-bounded block scores (RBS)" page: the block estimator of
 * "The idea", radius_bounded_block_scores and relative_block_mask of "What
 * mlx-arsenal ships", and the union of the recipe), 64-token blocks.
 *
 *   block_mask  [out] uint8 (B, Hq, ceil(Sq/64), ceil(Sk/64)) device array:
 *               2 = keep the block, 0 = skip it; pass it to attn_fwd_flex with
 *               block_mask_per_head = 1.
 *   base_scores, rescue_scores [out] float32, same shape, or NULL: the log
 *               block scores log sum_t exp(l_t) over the query block's tokens,
 *               l_base = <q, c> / sqrt(D), l_rescue = (<q, c> + |q| r beta) /
 *               sqrt(D), c / r the key block's centroid / radius, beta =
 *               clip((r - r_low) / (r_high - r_low), 0, 1) with r_low / r_high
 *               the median / 90th percentile of the KV head's block radii.
 *   Q (B, Hq, Sq, D), K (B, Hkv, Sk, D) bf16 device arrays (GQA: query head h
 *               scores the blocks of KV head h / (Hq / Hkv)).
 *   A block is kept when base >= row max + ln alpha_base, or rescue >= row max
 *   + ln alpha_rescue, or |qb - kb| < diagonal (the page uses 0.22, 0.18, 1).
 * Limits: Sk <= 131072, D in {64, 128}.  Allocates a stream-ordered workspace
 * of B * Hkv * ceil(Sk/64) * (D + 2) floats.
 */
attn_status_t attn_rbs_block_mask(uint8_t *block_mask, float *base_scores, float *rescue_scores,
                                  const void *Q, const void *K, int B, int Hq, int Hkv, int Sq,
                                  int Sk, int D, float alpha_base, float alpha_rescue,
                                  int diagonal, void *stream);

/*
 * attn_block_mask_build -- the page's build_block_mask (Tylo.jl "Primitives"
 * page, entry `build_block_mask`, TILE_M = TILE_N = 64) on the host.
 *
 *   out   [out] host uint8 (ceil(Sq/64), ceil(Sk/64)), caller-owned.  Block
 *         (qb, kb) gets 0 if keep is false for every (query row, key) pair of
 *         the block, 2 if it is true for every pair, 1 otherwise (pairs past
 *         Sq or Sk are not part of a block).
 *   keep  predicate on (q, kv): q = input_pos + i is the absolute position of
 *         query row i, kv the key position; nonzero = attend.
 * Returns ATTN_ERR_NULL / ATTN_ERR_INVALID on bad arguments.
 */
attn_status_t attn_block_mask_build(uint8_t *out, int Sq, int Sk, int input_pos,
                                    int (*keep)(int q, int kv, void *ctx), void *ctx);

/*
 * attn_block_mask_document -- attn_block_mask_build for the predicate
 * "doc_q[i] == doc_kv[kv], and the causal / window rule of attn_fwd holds"
 * (DocumentMask combined with CausalMask / the sliding window), with host
 * arrays doc_q (Sq,) and doc_kv (Sk,).
 */
attn_status_t attn_block_mask_document(uint8_t *out, int Sq, int Sk, int input_pos, int causal,
                                       int window, const int32_t *doc_q, const int32_t *doc_kv);

/*
 * attn_decode -- split-KV (Flash-Decoding) attention of one new query token per
 * head and sequence against a KV cache.
 *
 * Defined by: Tylo.jl "Primitives" page, entry `decode_attention!` (one query
 * vector per head and sequence, the KV cache processed in n_splits parallel
 * slices, lengths = valid KV length per sequence); scale is the page's default
 * qk_scale = 1/sqrt(D) (entry `flex_attention!`).  Slice s of sequence b
 * covers keys [s*C, min((s+1)*C, lengths[b])) with C = 64 * ceil(ceil(
 * lengths[b]/64) / n_splits); each slice yields a partial output and its
 * log-sum-exp, and a second kernel merges the slices by their log-sum-exp.
 *
 *   O        [out] bf16 (B, Hq, D)
 *   Q        [in]  bf16 (B, Hq, D)
 *   K, V     [in]  bf16 caches (B, Hkv, S_cap, D)
 *   lengths  [in]  int32 (B,) device array, required.  Values above S_cap are
 *                  clamped and flagged ATTN_ERR_DEVICE_BOUNDS; values <= 0
 *                  give O = 0 for that sequence.
 *   n_splits 1..64.
 *   Sizes: B >= 0; Hq, Hkv >= 1, Hq % Hkv == 0, Hq / Hkv <= 16, Hkv <= 65535;
 *          S_cap >= 0; D in {64, 128}.
 *
 * The per-slice partial results live in a workspace of
 * B * Hq * n_splits * (D + 4) floats that the call allocates and frees in
 * stream order on `stream`, from a memory pool the library keeps per device
 * (memory freed to it stays reserved for later calls).
 */
attn_status_t attn_decode(void *O, const void *Q, const void *K, const void *V,
                          const int32_t *lengths, int n_splits, void *stream,
                          int B, int Hq, int Hkv, int S_cap, int D);

/*
 * attn_decode_paged -- attn_decode over a paged KV cache (vllm-mlx
 * "attention" page: MLXAttentionBackend.get_kv_cache_shape gives the cache
 * shape (num_blocks, block_size, num_kv_heads, head_size); MLXAttentionMetadata
 * carries seq_lens and block_tables).
 *
 *   O       [out] bf16 (B, Hq, D)
 *   Q       [in]  bf16 (B, Hq, D), one new token per sequence
 *   K_cache, V_cache [in] bf16 (num_blocks, block_size, Hkv, D)
 *   block_tables [in] int32 (B, max_blocks_per_seq) device array: key j of
 *           sequence b is row j % block_size of block block_tables[b][j /
 *           block_size].  Entries past a sequence's last block are not read.
 *   seq_lens [in] int32 (B,) device array: keys 0 .. seq_lens[b]-1 attend.
 *           Values above max_blocks_per_seq * block_size are clamped and
 *           flagged ATTN_ERR_DEVICE_BOUNDS, as is a block index outside
 *           0 .. num_blocks-1 (that block then reads as zeros).
 *   n_splits, scale (1/sqrt(D)), GQA rule, workspace and errors as attn_decode.
 *   block_size: a power of two >= 8.
 */
attn_status_t attn_decode_paged(void *O, const void *Q, const void *K_cache, const void *V_cache,
                                const int32_t *block_tables, const int32_t *seq_lens, int n_splits,
                                void *stream, int B, int Hq, int Hkv, int num_blocks,
                                int block_size, int max_blocks_per_seq, int D);

/*
 * attn_decode_noalloc -- attn_decode for callers that cannot allocate device
 * memory.  The pages have no counterpart: it is attn_decode with a different
 * home for the per-slice workspace.
 *
 * Who needs it: attn_decode allocates and frees its workspace (stream
 * ordered, from the library's pool) on every call.  A serving loop that reserves all of its device memory up front and
 * forbids allocation afterwards (an allocation can fail once the memory is
 * spoken for, and its latency is not bounded), or a program whose device
 * memory belongs to another allocator, cannot let the library allocate.  This
 * entry point allocates nothing: it runs the same kernels with the workspace
 * in a fixed 16 MiB device array compiled into the library.
 *
 * Arguments, layouts, results and errors: as attn_decode, plus
 * ATTN_ERR_SCRATCH_LIMIT, returned before anything is enqueued, when the
 * workspace B * Hq * n_splits * (D + 4) * 4 bytes exceeds 16 MiB
 * (16777216 bytes; e.g. B 64, Hq 32, n_splits 8, D 128 needs 8.65 MB).
 *
 * Sharing rules: every GPU that loads the library holds the 16 MiB array until
 * the process exits, and all calls on one device share it.  Calls that can
 * overlap on the GPU (other streams, unordered host threads) race on it; issue
 * them on one stream or otherwise order them.  The array keeps the last call's
 * contents; nothing in it needs to start at zero.  The first call on a device,
 * made while that device is current, looks up the array's device address
 * (cudaGetSymbolAddress); make that first call before any stream capture.
 */
attn_status_t attn_decode_noalloc(void *O, const void *Q, const void *K, const void *V,
                                  const int32_t *lengths, int n_splits, void *stream,
                                  int B, int Hq, int Hkv, int S_cap, int D);

/*
 * attn_decode_sinks, attn_decode_paged_sinks -- attn_decode and attn_decode_paged of a
 * model with a sliding window and sinks.  The query is the last cached token, position
 * lengths[b] - 1, so it sees the keys
 *   j < lengths[b]  with  j >= lengths[b] - window  or  j < sinks.
 * Cache rows of other keys never reach O, whatever they hold; in the paged cache, entries
 * of block_tables for pages without a visible key may hold anything (attn_cache_free
 * leaves -1 there), and those pages are not read.
 * Arguments and errors as attn_decode / attn_decode_paged; window >= 1, sinks >= 0;
 * n_splits 0..64, 0 = chosen by the library from the sizes; S_cap, or
 * max_blocks_per_seq * block_size, at most 2^30.  Up to 8 slices need no workspace.
 */
attn_status_t attn_decode_sinks(void *O, const void *Q, const void *K, const void *V,
                                const int32_t *lengths, int window, int sinks, int n_splits,
                                void *stream, int B, int Hq, int Hkv, int S_cap, int D);
attn_status_t attn_decode_paged_sinks(void *O, const void *Q, const void *K_cache,
                                      const void *V_cache, const int32_t *block_tables,
                                      const int32_t *seq_lens, int window, int sinks,
                                      int n_splits, void *stream, int B, int Hq, int Hkv,
                                      int num_blocks, int block_size, int max_blocks_per_seq,
                                      int D);

/*
 * attn_tree_paged -- attention of a tree of drafted tokens over a paged KV cache
 * (speculative decoding: T drafts of each sequence checked in one pass).
 *
 *   O        [out] bf16 (B, Hq, T, D)
 *   Q        [in]  bf16 (B, Hq, T, D)
 *   K_cache, V_cache, block_tables [in] as attn_decode_paged.  The drafts' keys and values
 *            already stand in the pages: draft i of sequence b at position
 *            context_lens[b] + i (attn_cache_append writes them).
 *   context_lens [in] int32 (B,): committed tokens of each sequence.
 *   parents  [in] int32 (B, T): draft i continues draft parents[b][i], or the context
 *            for -1.  Every parent comes before its child (-1 <= parents[b][i] < i).
 *   draft_lens [in] int32 (B,) or NULL (= T): drafts i >= draft_lens[b] do not exist;
 *            their rows of O are +0.0, whatever Q holds there.
 *
 * Draft i sees every key before context_lens[b], itself and its ancestors; scale is
 * 1/sqrt(D).  A negative context length counts as 0; lengths past the table are clamped,
 * a parent outside its range counts as -1, and a page outside the pool reads as zeros;
 * each is flagged ATTN_ERR_DEVICE_BOUNDS.  Cache rows at or past context_lens[b] +
 * draft_lens[b] never reach O; those before it must hold finite values.
 *   Sizes: B >= 0; T 0..256; Hq, Hkv >= 1, Hq % Hkv == 0, Hq / Hkv <= 16;
 *          max_blocks_per_seq >= 1; block_size a power of two >= 8; D in {64, 128};
 *          max_blocks_per_seq * block_size at most 2^30.
 * Allocates a stream-ordered workspace (partial results of the sequences that several
 * SMs share, up to 39 MB, and B + 1 integers).
 */
attn_status_t attn_tree_paged(void *O, const void *Q, const void *K_cache, const void *V_cache,
                              const int32_t *block_tables, const int32_t *context_lens,
                              const int32_t *parents, const int32_t *draft_lens, void *stream,
                              int B, int Hq, int Hkv, int T, int num_blocks, int block_size,
                              int max_blocks_per_seq, int D);

/*
 * Operators on a paged KV cache
 * -----------------------------
 * The cache is attn_decode_paged's: pools (num_blocks, block_size, Hkv, D) and
 * block_tables int32 (R, max_blocks_per_seq), -1 where a sequence has no page.  A
 * serving loop keeps one table and one ref_counts for all layers and one pair of pools
 * per layer: append, compact and copy_blocks work on a layer's pools, fork, extend and
 * free on the table.
 *   ref_counts int32 (num_blocks): how many table entries name each page.  A page is
 *   free when its count is 0; fork and extend hand out the lowest free pages first, so
 *   their results depend on their arguments alone.  Like every tensor, ref_counts is
 *   16-byte aligned; the other int32 arrays need 4 bytes.
 * block_size is a power of two >= 8, max_blocks_per_seq >= 1, num_blocks >= 1, and
 * num_blocks * block_size and max_blocks_per_seq * block_size below 2^31.  Calls that
 * share a table, counts or pages are to be ordered by the caller (one stream).
 */

/*
 * attn_cache_append -- write new rows of keys and values to their pages.
 *   K_new, V_new [in] bf16 (B, Hkv, T, D) (the layout attn_fwd reads)
 *   start  [in] int32 (B,): row t of sequence b goes to position start[b] + t
 *   n_new  [in] int32 (B,) or NULL (= T): rows t >= n_new[b] are not written.
 * A row whose position lies outside the table, or on an entry without a page of the
 * pool, is not written and flagged ATTN_ERR_DEVICE_BOUNDS, as is n_new[b] > T (clamped).
 * Two rows of one call may not go to the same place (pages shared by two sequences).
 */
attn_status_t attn_cache_append(void *K_cache, void *V_cache, const void *K_new,
                                const void *V_new, const int32_t *block_tables,
                                const int32_t *start, const int32_t *n_new, void *stream,
                                int B, int Hkv, int T, int num_blocks, int block_size,
                                int max_blocks_per_seq, int D);

/*
 * attn_cache_compact -- move the rows that are kept to the front, in place: position
 * base[b] + k takes the keys and values of position base[b] + keep[b][k],
 * k < n_keep[b] (the accepted path of a tree of drafts; the rows a pruned cache keeps).
 *   base   [in] int32 (B,)
 *   keep   [in] int32 (B, A), strictly increasing, >= 0 over its first n_keep[b] entries
 *   n_keep [in] int32 (B,) or NULL (= A); values above A are clamped and flagged.
 * Rows past base[b] + n_keep[b] are left as they are.  A sequence whose list is not
 * increasing, leaves the table, or touches an entry without a page of the pool is left
 * untouched and flagged ATTN_ERR_DEVICE_BOUNDS.  Rows that two sequences share may not be
 * moved.
 */
attn_status_t attn_cache_compact(void *K_cache, void *V_cache, const int32_t *block_tables,
                                 const int32_t *base, const int32_t *keep,
                                 const int32_t *n_keep, void *stream, int B, int Hkv, int A,
                                 int num_blocks, int block_size, int max_blocks_per_seq, int D);

/*
 * attn_cache_copy_blocks -- page dst[i] takes the contents of page src[i], i < N, in both
 * pools.  A pair with a negative entry is no pair.  A pair is skipped and flagged
 * ATTN_ERR_DEVICE_BOUNDS when a page is outside the pool, when its source is another
 * pair's destination, or when a later pair names the same destination.  N <= 65536; every
 * pair is compared with all others, so a list of tens of thousands costs milliseconds.
 */
attn_status_t attn_cache_copy_blocks(void *K_cache, void *V_cache, const int32_t *src,
                                     const int32_t *dst, void *stream, int N, int num_blocks,
                                     int block_size, int Hkv, int D);

/*
 * attn_cache_fork -- sequences that continue others: row children[n] of the table becomes
 * a copy of row parents[n] up to its length.  Whole pages are shared (their counts rise by
 * one); a part-filled last page is not: the child gets a free page for it (count 1), and
 * the pair of pages goes to copy_src[n], copy_dst[n] (-1, -1 without one), for
 * attn_cache_copy_blocks on every layer.  The rest of the child's row is -1, and
 * seq_lens[children[n]] = seq_lens[parents[n]].
 *   block_tables [in/out] int32 (R, max_blocks_per_seq), ref_counts [in/out],
 *   seq_lens [in/out] int32 (R,), parents, children [in] int32 (N,),
 *   copy_src, copy_dst [out] int32 (N,).
 * The child's row is overwritten: give back what it held first (attn_cache_free).  A pair
 * with a negative entry is no pair.  A pair is skipped and flagged ATTN_ERR_DEVICE_BOUNDS
 * when a row is outside the table, when its child is also a parent, or the child of an
 * earlier pair.  Free pages go to the pairs in order; a pair that gets none keeps -1
 * there and the call flags ATTN_ERR_NO_PAGES (also over a DEVICE_BOUNDS that no one has
 * read yet).  N <= 65536; every pair is compared with all others.
 * A child without its last page is the one whose seq_lens is not a multiple of block_size
 * and whose table entry at seq_lens / block_size is negative (its copy_src and copy_dst
 * are -1).  Its last tokens are nowhere: attention flags the missing page, but
 * attn_cache_extend would put an empty page there and its old rows would be read.  Free
 * its row and fork it again when there are pages.  Entries that the parent itself lacks
 * are missing in the child too, without a flag.
 */
attn_status_t attn_cache_fork(int32_t *block_tables, int32_t *ref_counts, int32_t *seq_lens,
                              const int32_t *parents, const int32_t *children,
                              int32_t *copy_src, int32_t *copy_dst, void *stream, int N, int R,
                              int num_blocks, int block_size, int max_blocks_per_seq);

/*
 * attn_cache_extend -- pages for the next tokens: in each row r, the empty (negative)
 * entries from the page of position from_lens[r] to the last page that to_lens[r] tokens
 * need get free pages (count 1), rows in order, entries in order.  Entries that hold a
 * page keep it.  to_lens[r] past the table is clamped and flagged
 * ATTN_ERR_DEVICE_BOUNDS; entries for which no page is left stay as they are and the call
 * flags ATTN_ERR_NO_PAGES (over DEVICE_BOUNDS, as fork).  A page comes with the rows that it
 * held before; the caller writes those that it reads (attn_cache_append).
 *   block_tables, ref_counts [in/out], from_lens, to_lens [in] int32 (R,).
 * R * max_blocks_per_seq is below 2^31.
 */
attn_status_t attn_cache_extend(int32_t *block_tables, int32_t *ref_counts,
                                const int32_t *from_lens, const int32_t *to_lens, void *stream,
                                int R, int num_blocks, int block_size, int max_blocks_per_seq);

/*
 * attn_cache_free -- give back the pages of table entries first[n] .. last[n]-1 of row
 * rows[n], n < N: the entries become -1 and their pages' counts fall by one (a whole
 * sequence; the pages behind a rejected draft; those that left a sliding window).  Empty
 * entries are passed over, ranges are cut to the table, and a negative row names none.
 * A row or page out of range, or a page whose count is already 0 (which stays 0), is
 * flagged ATTN_ERR_DEVICE_BOUNDS.
 */
attn_status_t attn_cache_free(int32_t *block_tables, int32_t *ref_counts, const int32_t *rows,
                              const int32_t *first, const int32_t *last, void *stream, int N,
                              int R, int num_blocks, int max_blocks_per_seq);

/* Human-readable name of a status code (static storage, never NULL). */
const char *attn_status_string(attn_status_t status);

/*
 * attn_last_device_status -- synchronise `stream`, then return and clear the
 * status word that kernels of this library set on the current device
 * (ATTN_OK if none did).  The word keeps the first status set since it was last
 * read, except that ATTN_ERR_NO_PAGES replaces ATTN_ERR_DEVICE_BOUNDS.  Returns ATTN_ERR_CUDA if the synchronisation failed.
 */
attn_status_t attn_last_device_status(void *stream);

/*
 * attn_check_bounded_wait -- diagnostic for the library's bounded waits.
 * Launches one block that waits on a barrier nobody completes, with a limit
 * of `limit_us` microseconds (1..2000000), through the same wait routine the
 * attention kernels use.  The kernel gives up, records ATTN_ERR_TIMEOUT in
 * the device status word and returns; read it with attn_last_device_status.
 * No page defines this; it exists to test the failure path without a hang.
 */
attn_status_t attn_check_bounded_wait(int limit_us, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GQA_ATTN_H */
