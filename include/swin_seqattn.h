/*
 * swin_seqattn.h -- C ABI of libswinwattn.so, second part: attention along a
 * token sequence (sliding window with sink tokens, forward and backward) and
 * the paged key-value cache that serves it token by token.
 *
 * It is the one-dimensional, causal counterpart of the windows of
 * swin_wattn.h: the tokens of a rollout attend to the recent tokens of their
 * own sequence and to its first ones. Status codes, element types, ownership,
 * streams and the device status word (swin_wattn_poll_status) are those of
 * swin_wattn.h: every data pointer is device memory of the current device
 * owned by the caller, nothing is allocated, nothing is synchronised, and two
 * calls in flight at once must not share a workspace (calls, or captured
 * graphs, that follow one another on a stream may). The first 256 bytes of a
 * workspace are zeroed by the caller once, before its first use: they hold the
 * status word; the rest may hold anything. Every call can be
 * captured into a CUDA graph; lengths, counts and page tables are read on the
 * device when it runs.
 *
 * ---- attention along a sequence ---------------------------------------------
 * Query head h reads kv head h / (heads / kv_heads). Key j is visible to
 * query i of a sequence of n tokens when
 *     j <= i < n  and  (window == 0  or  i - j < window  or  j < sinks).
 * a_ij = q_i.k_j / sqrt(head_dim), lse_i = log sum_j exp(a_ij) over the
 * visible keys, P_ij = exp(a_ij - lse_i), o_i = sum_j P_ij v_j. The backward
 * returns, with dP_ij = dO_i.v_j, D_i = dO_i.o_i and dS_ij = P_ij (dP_ij - D_i),
 *     dq_i = sum_j dS_ij k_j / sqrt(head_dim),
 *     dk_j = sum_i dS_ij q_i / sqrt(head_dim),  dv_j = sum_i P_ij dO_i,
 * the last two summed over the query heads that share the kv head.
 * `lengths` (int32 [B], may be NULL: S tokens each) gives each sequence's n;
 * a value below 0 counts as 0, one above S as S. Tokens at and beyond n are
 * padding: what q, k, v, dout, out and lse hold there is not used, NaN
 * included, and their out, lse, dq, dk and dv are written as zeros.
 * A masked key has no influence on a row, whatever it holds: a NaN or an
 * infinity reaches only the rows that see it. (Rows that such a value would
 * have spoiled through a shared tile are computed once more, one at a time;
 * results are exact, the call is slower.)
 * Repeated calls give identical bits.
 *
 * Layouts: q [B, S, heads, head_dim], k and v [B, S, kv_heads, head_dim] of
 * `dtype`, each token's heads contiguous and tokens q_stride (q, dq) or
 * kv_stride (k, v, dk, dv) elements apart, so that q, k and v may be parts of
 * one projection's output; sequences S tokens apart. out and dout
 * [B, S, heads, head_dim] contiguous, lse [B, S, heads] fp32. Outputs must
 * not overlap inputs or one another (parts of one buffer that interleave
 * without sharing an element do not overlap).
 */
#ifndef SWIN_SEQATTN_H
#define SWIN_SEQATTN_H

#include "swin_wattn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* B, S >= 1; heads a multiple of kv_heads >= 1; 8 <= head_dim <= 256, a
 * multiple of 8; window, sinks >= 0 (window 0: every earlier token);
 * q_stride, kv_stride 0 (contiguous) or at least heads (kv_heads) * head_dim
 * and a multiple of 16 bytes; S <= 2^30, B * S < 2^31. flags: SWIN_FLAG_FORCE_GENERIC
 * and SWIN_FLAG_TEST_TIMEOUT. */
typedef struct swin_seqattn_desc {
  int32_t B, S;
  int32_t heads, kv_heads, head_dim;
  int32_t window, sinks;
  int32_t dtype; /* enum swin_wattn_dtype */
  int32_t flags; /* enum swin_wattn_flags */
  int32_t q_stride, kv_stride;
} swin_seqattn_desc;

/* Kernel family: 1 = tcgen05/TMA kernels (bf16, head_dim up to 128), 0 =
 * portable kernels (fp32 and other head sizes). Negative status for an
 * invalid description. Host only. */
int swin_seqattn_path(const swin_seqattn_desc* desc);

/* Bytes of workspace (256-byte aligned) the forward and backward need. */
int swin_seqattn_workspace_size(const swin_seqattn_desc* desc, size_t* bytes);

/* Forward. `lse` may be NULL. Pointers 16-byte aligned (lengths: 4). */
int swin_seqattn_fwd(const swin_seqattn_desc* desc, const void* q, const void* k, const void* v,
                     const int32_t* lengths, void* out, float* lse, void* workspace,
                     size_t workspace_bytes, void* stream);

/* Backward from the forward's out and lse; dq, dk and dv are overwritten. */
int swin_seqattn_bwd(const swin_seqattn_desc* desc, const void* q, const void* k, const void* v,
                     const int32_t* lengths, const void* out, const float* lse, const void* dout,
                     void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes,
                     void* stream);

/* ---- paged key-value cache -----------------------------------------------------
 * k_cache and v_cache: [num_pages, kv_heads, page_size, head_dim] of `dtype`.
 * page_table: int32 [B, max_pages]; position p of sequence b is row
 * p % page_size of page page_table[b, p / page_size]. lengths: int32 [B], the
 * tokens of each sequence, 0 .. max_pages * page_size (values outside count as
 * the nearest bound). Entries of the table at and beyond a sequence's last page
 * are not read. A page id outside 0 .. num_pages - 1 where one is needed is
 * not followed: its positions are left out of the attention and of the
 * copies, and the workspace's status word becomes SWIN_ERR_INVALID_ARG, which
 * swin_wattn_poll_status reports. Weights: fp32 [B, kv_heads, max_pages *
 * page_size].
 *
 * B, page_size, num_pages, max_pages >= 1; page_size <= 65536; heads and
 * head_dim as above; window, sinks >= 0. q_stride and kv_stride: elements from
 * one token to the next in q (decode) and in the new keys and values (decode,
 * append); 0 = contiguous. At most 1024 query heads to a kv head;
 * B * kv_heads * max_pages * page_size at most 2^40, max_pages * page_size at
 * most 2^30 and num_pages * kv_heads * page_size * head_dim at most 2^48. Outputs must not overlap inputs or one another, except where
 * a call says so. */
enum swin_kvcache_flags {
  SWIN_FLAG_KV_WEIGHTS = 1 << 8 /* decode calls will accumulate weights: the workspace also
                                   holds the step's logits, 4 bytes per query head and
                                   visible position */
};
typedef struct swin_kvcache_desc {
  int32_t B;
  int32_t heads, kv_heads, head_dim;
  int32_t page_size, num_pages, max_pages;
  int32_t window, sinks;   /* decode: as in swin_seqattn_desc; evict: sinks are always kept */
  int32_t recent, budget;  /* evict */
  int32_t dtype, flags;    /* enum swin_wattn_dtype, swin_kvcache_flags */
  int32_t q_stride, kv_stride;
} swin_kvcache_desc;

/* Bytes of workspace (256-byte aligned) for any of the calls below. */
int swin_kvcache_workspace_size(const swin_kvcache_desc* desc, size_t* bytes);

/* Writes new tokens into the cache. k, v: [B, T, kv_heads, head_dim], tokens
 * kv_stride elements apart, sequences T tokens apart; T * kv_heads * head_dim
 * at most 2^31, that times B at most 2^38. `counts` (int32 [B], NULL:
 * T each; clamped to 0 .. T): the first counts[b] tokens of sequence b are
 * written, to positions lengths[b] - counts[b] .. lengths[b] - 1: `lengths`
 * already counts them. A count above the length writes only the tokens whose
 * position is not negative and sets the status word as a bad page does.
 * No other row of the cache is touched. Two positions that share a page row
 * (the same page twice) end with one or the other's values. */
int swin_kvcache_append(const swin_kvcache_desc* desc, int32_t T, const void* k, const void* v,
                        const int32_t* counts, const int32_t* lengths, const int32_t* page_table,
                        void* k_cache, void* v_cache, void* workspace, size_t workspace_bytes,
                        void* stream);

/* Attention of one query token per sequence, at position lengths[b] - 1, over
 * the cache: q and out [B, heads, head_dim] (q's tokens q_stride apart), lse
 * [B, heads] fp32 or NULL. k_new, v_new [B, kv_heads, head_dim] (kv_stride
 * apart; both or neither NULL): the token's own key and value, attended to and
 * written to position lengths[b] - 1 of the cache; NULL when the cache already
 * holds them. An empty sequence (and one whose every
 * visible page is bad) gets out = 0 and lse = -inf.
 * new_weights (may be NULL) receives weights + the sum over the kv head's query
 * heads of this step's P for every position below the length (positions that
 * the window hides keep their weight, nothing beyond the length is written);
 * `weights` may be the same buffer, and must be given with new_weights. Both
 * need SWIN_FLAG_KV_WEIGHTS in the description (it sizes the workspace).
 * Work is split over the cache's length and joined in a fixed order: repeated
 * calls give identical bits. Sequences may share pages, except a page that
 * receives a new token. */
int swin_kvcache_decode(const swin_kvcache_desc* desc, const void* q, const void* k_new,
                        const void* v_new, const int32_t* lengths, const int32_t* page_table,
                        void* k_cache, void* v_cache, const float* weights, float* new_weights,
                        void* out, float* lse, void* workspace, size_t workspace_bytes,
                        void* stream);

/* Evicts positions by accumulated weight, each kv head on its own. A sequence
 * of n <= budget tokens keeps all of them; otherwise it keeps its first
 * `sinks`, its last `recent` (sinks + recent <= budget) and the budget - sinks
 * - recent of the rest that have the largest weights (ties: the lowest
 * position; NaN counts below every number; -0 equals +0), in their order. The
 * kept rows are copied within k_cache and v_cache to the pages of
 * dst_page_table ([B, max_pages], at least ceil(min(n, budget) / page_size)
 * valid entries), which must not be pages that page_table names below the
 * lengths: the old pages stay as they are and are the caller's to free, so
 * sequences may share them. new_weights [B, kv_heads, max_pages * page_size]
 * (not the same buffer as weights) receives the kept weights and zeros behind
 * them, new_lengths [B] (not lengths itself) the kept counts, kept (int32 [B, kv_heads, budget],
 * may be NULL) the kept positions, -1 behind the last. 1 <= budget <=
 * max_pages * page_size, recent >= 0. */
int swin_kvcache_evict(const swin_kvcache_desc* desc, const float* weights,
                       const int32_t* lengths, const int32_t* page_table,
                       const int32_t* dst_page_table, void* k_cache, void* v_cache,
                       float* new_weights, int32_t* new_lengths, int32_t* kept, void* workspace,
                       size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SWIN_SEQATTN_H */
