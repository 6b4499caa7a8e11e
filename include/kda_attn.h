/*
 * kda_attn.h -- C ABI of the operators that a hybrid stack's attention layers
 * need beside KDA on GB300 (sm_103a): norms of queries and keys with the
 * position's rotation, the paged key-value cache, attention of new tokens over
 * it, and the verification of drafted tokens.
 *
 * The conventions are those of kda.h and kda_layer.h: the caller owns every
 * buffer, nothing is allocated, calls are asynchronous on `stream`, errors that
 * the host can see return before anything is launched, activations may be
 * column slices of a wider tensor (a token stride in elements, 0 = dense; any
 * base that is a multiple of the element size), and 16-byte alignment of base
 * and stride selects the wide loads.  Where `workspace` is optional a NULL skips
 * the report of errors found on the device; otherwise its first word holds the
 * call's device status after the call.  Outputs alias no input unless an entry
 * point says so.
 */
#ifndef KDA_ATTN_H_
#define KDA_ATTN_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Norms of queries and keys with the position's rotation.  Per token and head
 * of d channels:
 *
 *     n = x / sqrt(mean(x^2) + eps) weight       (n = x when weight is NULL)
 *     (a, b) -> (a cos f - b sin f, a sin f + b cos f),   f = position freqs[i]
 *
 * for the rot / 2 pairs of the first rot channels: (i, i + rot / 2), or with
 * `interleaved` (2i, 2i + 1).  The other channels keep n.  Angles are reduced
 * to within 2^-31 of a turn for all frequencies and positions (a frequency over
 * 2 pi counts in multiples of 2^-64).  Evaluated in float32, each output rounded
 * once.
 * ---------------------------------------------------------------------- */
typedef struct {
  int64_t tokens;       /* >= 0 */
  int32_t q_heads;      /* heads of q per token, 1 .. 65536 */
  int32_t k_heads;      /* heads of k per token, 0 .. 65536 (0: no k) */
  int32_t d;            /* channels per head, even, 2 .. 256 */
  int32_t rot;          /* rotated channels, even, 0 .. d */
  kda_dtype dtype;      /* q, k, their outputs and gradients */
  int32_t interleaved;
  float eps;
  int64_t ldq, ldk;     /* elements between tokens of q and k; 0 = dense */
} kda_qknorm_shape;

/* q [tokens,q_heads,d], k [tokens,k_heads,d], positions int32 [tokens] (any
 * sign), freqs float64 [rot/2] (radians per position, finite, at most 2^20 in size),
 * q_weight and k_weight f32 [d] or NULL, q_out and k_out dense.  q_out may be
 * q and k_out may be k where those are dense. */
kda_status kda_qknorm_fwd(const kda_qknorm_shape* s, const void* q, const void* k,
                          const int32_t* positions, const double* freqs, const float* q_weight,
                          const float* k_weight, void* q_out, void* k_out, void* stream);

/* Gradients of sum(q_out dq_out) + sum(k_out dk_out).  dq_out, dk_out, dq, dk
 * dense; dq_weight, dk_weight f32 [d], each NULL when its weight is absent or
 * its gradient is not wanted; positions and freqs have none.  Sums over rows
 * are taken in a fixed order.  workspace: kda_qknorm_bwd_workspace_size(s)
 * bytes, 256-byte aligned. */
size_t kda_qknorm_bwd_workspace_size(const kda_qknorm_shape* s);
kda_status kda_qknorm_bwd(const kda_qknorm_shape* s, const void* q, const void* k,
                          const void* dq_out, const void* dk_out, const int32_t* positions,
                          const double* freqs, const float* q_weight, const float* k_weight,
                          void* dq, void* dk, float* dq_weight, float* dk_weight, void* workspace,
                          size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * The paged key-value cache.  Keys and values each live in a pool of pages
 * [num_pages, heads, page, d].  A sequence's token at place p is row p % page
 * of the page that its row of the table, pages [N, max_pages] int32, names at
 * p / page.  A cache of 8-bit codes (KDA_CACHE_E4M3, KDA_CACHE_INT8) comes
 * with a byte per row, scale [num_pages, heads, page]: a row's values are
 * code 2^(byte - 127), with the smallest such power of two (2^-126 at least)
 * that brings the row's largest size into the type's range (448, 127); codes
 * are rounded to nearest, ties to even.  Scaling by a power of two is exact, so
 * the codes are defined bit by bit.  A row that holds an infinity or a NaN is
 * kept as byte 255 and codes 0, and reads back as NaN.
 * ---------------------------------------------------------------------- */
typedef enum {
  KDA_CACHE_F32 = 0,
  KDA_CACHE_BF16 = 1,
  KDA_CACHE_E4M3 = 2,
  KDA_CACHE_INT8 = 3
} kda_cache_dtype;

typedef struct {
  int32_t B;            /* fixed length: sequences.  Packed: must be 1. */
  int32_t T;            /* tokens per sequence (fixed) or in total (packed), >= 0 */
  int32_t num_seqs;     /* packed: number of sequences; ignored when cu_seqlens is NULL */
  int32_t heads, d;     /* key-value heads, 1 .. 65536; channels 64 or 128 */
  int32_t page;         /* tokens per page, a power of two up to 65536 */
  int32_t max_pages;    /* columns of the page table, >= 1 */
  int32_t num_pages;    /* pages in the pools, >= 1 */
  kda_dtype dtype;      /* k and v */
  kda_cache_dtype cache;
  int64_t ldk, ldv;     /* elements between tokens of k and v (written only); 0 = dense */
  int64_t ldpage;       /* elements between pages of both pools, a multiple of 16 bytes;
                           0 = heads page d.  The scales are dense. */
} kda_cache_shape;

/* Write.  lens int32 [N]: tokens of each sequence after the write, so that the
 * n tokens that the call brings for a sequence go to places lens - n .. lens - 1.
 * Tokens whose place is below 0 (an idle row of a padded batch has lens 0) are
 * left out; a place past the table or a page that is not in the pool is left
 * out and reported (KDA_ERR_INVALID_ARG), malformed cu_seqlens are reported
 * (KDA_ERR_BAD_SEQLENS); every access stays inside the buffers.  A row in which
 * two tokens of one call meet is undefined.  k_cache, v_cache, k_scale and
 * v_scale are 16-byte aligned; the scales are given exactly with 8-bit caches.
 * workspace: optional, >= 256 bytes, 256-byte aligned. */
kda_status kda_cache_write(const kda_cache_shape* s, const void* k, const void* v,
                           const int32_t* cu_seqlens, const int32_t* pages, const int32_t* lens,
                           void* k_cache, void* v_cache, uint8_t* k_scale, uint8_t* v_scale,
                           void* workspace, size_t workspace_bytes, void* stream);

/* Read the same places back: k and v [B,T,heads,d] dense (either may be NULL)
 * get the tokens lens - n .. lens - 1 of each sequence, rounded to dtype where
 * that is narrower than the cache.  Rows whose place is below 0, past the table
 * or on a page that is not in the pool are zeros (the latter two reported);
 * rows behind the last sequence of a packed batch stay as they are. */
kda_status kda_cache_read(const kda_cache_shape* s, const int32_t* cu_seqlens,
                          const int32_t* pages, const int32_t* lens, const void* k_cache,
                          const void* v_cache, const uint8_t* k_scale, const uint8_t* v_scale,
                          void* k, void* v, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Attention of the newest T = 1..8 tokens of each of B sequences over its paged
 * cache, in which their own keys and values are already written.  Token t
 * stands at place lens - T + t and sees the places up to its own, with `window`
 * only the last `window` of them:
 *
 *     out = sum_j softmax_j(scale q . k_j) v_j,    lse = log sum_j exp(scale q . k_j)
 *
 * Query head h reads key-value head h / (q_heads / kv_heads).  A token that
 * sees nothing (its place is below 0) gets zeros and lse = -inf.  A row of the
 * cache that a token does not see does not touch it, whatever it holds.  A value
 * that it sees and that is infinite gives its channel that infinity (of both
 * signs: NaN), whatever its weight, and a NaN NaN; a query or a seen key that is
 * not finite may make the rows of that query, or all that see the key, NaN.
 * ---------------------------------------------------------------------- */
typedef struct {
  int32_t B, T;         /* sequences >= 0; tokens 1 .. 8 */
  int32_t q_heads, kv_heads; /* q_heads a multiple of kv_heads, at most 65536 */
  int32_t d;            /* 64 or 128 */
  int32_t page, max_pages, num_pages; /* as kda_cache_shape */
  kda_dtype dtype;      /* q and out */
  kda_cache_dtype cache; /* the type of q, or 8 bits */
  float scale;
  int32_t window;       /* 0 = all */
  int64_t ldq;          /* elements between tokens of q; 0 = dense */
  int64_t ldpage;       /* as kda_cache_shape */
} kda_attn_shape;

/* q [B,T,q_heads,d], out the same, dense; lse f32 [B,T,q_heads] or NULL.
 * Places that a token would see on a page that is not in the pool count as unseen
 * and are reported (KDA_ERR_INVALID_ARG), as is a lens past the table (the places
 * that it has are seen); the table's other entries may hold anything.  The keys are
 * split over the device by equal numbers of tiles and the parts joined in a fixed
 * order: results repeat bit for bit on one device.  Sums and statistics are float32.
 * With bf16 the scores are exact products in float32, and the weights enter the
 * second product with 16 bits over a bf16 cache and over one of 8 bits with 22 up to
 * 8 query rows (T q_heads / kv_heads) and with 11 from 9 on; with float32 products
 * keep 22 bits over an 8-bit cache and 24 over a float32 one.  Over 8 bits what counts
 * for a query row is its weight times the value row's power of two: 11 (22) bits for
 * products down to 2^-23 of its largest, 2^-34 of that for those below.  Where all
 * that it sees has powers below 2^-87 (values below 2^-78), bits are lost.
 * workspace: 256-byte aligned, kda_attn_workspace_size(s) bytes; where those are 256
 * they hold the status alone and may be left out (NULL, 0). */
size_t kda_attn_workspace_size(const kda_attn_shape* s);
kda_status kda_attn_step(const kda_attn_shape* s, const void* q, const void* k_cache,
                         const void* v_cache, const uint8_t* k_scale, const uint8_t* v_scale,
                         const int32_t* pages, const int32_t* lens, void* out, float* lse,
                         void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Verification of drafted tokens.  Per sequence, with the target's
 * probabilities p [K+1,V] after each draft, the draft's own q [K,V] (NULL: each
 * draft was certain, q = 1 at its token) and random numbers u [K+1] in [0, 1):
 * draft i is kept while u_i q_i(d_i) < p_i(d_i) (compared exactly).  Behind the
 * n kept ones one more token is drawn from
 *
 *     w = max(p_n - q_n, 0)    after a refusal (p_n itself where that is 0 throughout)
 *     w = p_n                  when every draft was kept
 *
 * as the first token whose running sum of w exceeds u_K of the whole.
 * Probabilities count in whole multiples of 2^-44 (rounded to nearest, below 0
 * and NaN as 0, above 1 as 1) and u_K in multiples of 2^-24 (rounded down): the
 * sums are exact, so the token does not depend on how they are split.
 * ---------------------------------------------------------------------- */
typedef struct {
  int32_t B;            /* sequences, >= 0 */
  int32_t K;            /* drafted tokens per sequence, 0 .. 31 */
  int32_t V;            /* tokens of the vocabulary, 1 .. 2^19 - 1 */
  kda_dtype dtype;      /* p and q */
} kda_verify_shape;

/* p [B,K+1,V], q [B,K,V] or NULL, drafts int32 [B,K], num_draft int32 [B] or
 * NULL (K): the drafts that a sequence has (its row p[num_draft] is the last),
 * -1 for an idle row of a padded batch.  u f32 [B,K+1], the last one for the
 * drawn token.  tokens int32 [B,K+1]: the kept drafts, the drawn token, then -1.
 * num_commit int32 [B]: n + 1, 0 for an idle row -- the tokens of the step
 * (the last known one and the kept drafts) whose state the step forms of KDA,
 * the convolution and the scan keep.  Reported as KDA_ERR_INVALID_ARG: a draft
 * outside the vocabulary (refused, as one of probability 0), a count outside
 * -1..K (an idle row), a row that has nothing to draw from (-1 in its place).
 * workspace: optional, >= 256 bytes, 256-byte aligned. */
kda_status kda_draft_verify(const kda_verify_shape* s, const void* p, const void* q,
                            const int32_t* drafts, const int32_t* num_draft, const float* u,
                            int32_t* tokens, int32_t* num_commit, void* workspace,
                            size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* KDA_ATTN_H_ */
