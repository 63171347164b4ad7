/*
 * tfserve.h - serving operators next to the paged attention of tfpaged.h: an
 * 8-bit KV cache (written, read back, attended to), attention of many streams
 * over shared prefixes, and the log probabilities of logit rows.
 *
 * They stand on the sources tfpaged.h names (TensorFold #1503 "lfm2_moe CUDA:
 * attention pages from the shared KV pool, and the prompt cache": streams
 * whose pages come from one pool, prefixes kept by the prompt cache, the
 * verify rows' argmax on the GPU); those pages give no layout or formula for
 * them, so the definitions below are this library's own.
 *
 * The conventions of tfpaged.h hold: device pointers except those named
 * *_host, no allocation, no synchronization, work enqueued on `stream`,
 * host-checkable errors returned before anything is launched, table errors
 * found on the device OR-ed into the caller's status word, segment tables of
 * tf_seg entries whose rows' keys are their stream's last ones.  Calls on one
 * stream order themselves; calls on different streams, or two replays of
 * captured graphs, must not overlap while they share a workspace or an output.
 */
#ifndef TFSERVE_H
#define TFSERVE_H

#include "tfpaged.h"

#if defined(__GNUC__)
#define TFS_API __attribute__((visibility("default")))
#else
#define TFS_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/*
 * A launch whose bounded wait gave up (TF_DEV_TIMEOUT in the status word) leaves
 * the rows of tf_paged_attn_q8 and tf_paged_attn_shared flagged NaN, as may any
 * later call while the caller has not cleared that bit.
 */

/* A given token lies outside [0, n_cols) (tf_logprob_rows). */
#define TF_DEV_BAD_TOKEN 0x20u

/* Code types of an 8-bit cache. */
enum { TF_KV_E4M3 = 1, TF_KV_INT8 = 2 };

/*
 * An 8-bit cache (a host struct of device pointers, read during a call).
 * Every (page, kv-head, slot) row of K and of V holds head_dim codes and one
 * scale byte e, which stands for 2^(e - 127); an element's value is
 * code * 2^(e - 127), the code an e4m3 number or a signed byte.  Bytes 27 to
 * 249 are scales; 255 marks a row that held a NaN or an infinity (its codes
 * are 0): a query that sees it is flagged.  A value is exact in bf16, so
 * attention over the cache and over its read-back are one attention.  (An
 * e4m3 NaN code under another scale byte, which no append writes, flags the
 * queries that see it and may flag other rows of its stream.)
 *
 *  k_codes, v_codes  u8 [n_pages][n_kv_heads][page_size][head_dim], 16-byte aligned
 *  k_scale, v_scale  u8 [n_pages][n_kv_heads][page_size], 16-byte aligned
 *
 * Supported: head_dim in {64, 128, 256}; page_size a power of two in [8, 1024].
 */
typedef struct {
    void *k_codes, *v_codes;
    uint8_t *k_scale, *v_scale;
    int32_t kv_type; /* TF_KV_E4M3 or TF_KV_INT8 */
    int32_t n_pages, page_size, n_kv_heads, head_dim;
} tf_q8_cache;

/*
 * tf_kv_append into an 8-bit cache: each stream's new rows are quantised as
 * they are written into their pages.  Row i of stream s is key
 * n_keys - n_rows + i, as for tf_kv_append, whose arguments, checks and errors
 * these are.
 *
 * Per (row, kv-head), for K and for V: amax = the row's largest magnitude, k =
 * the smallest integer >= -100 with amax <= Q * 2^k (Q = 448 for e4m3, 127 for
 * int8), scale byte k + 127, code = x * 2^-k rounded to nearest, ties to even.
 * Scaling by a power of two is exact, so the codes are those of the formula bit
 * for bit; an element is off by at most 2^-4 of itself (e4m3, above 2^(k-6)) or
 * by 2^(k-1) (int8).  A row holding a NaN or an infinity is stored as codes 0
 * and scale byte 255.  (A magnitude that rounds to 2^128 reads as infinity.)
 * Streams must not share the slots they write.  As a host table sizes the launch,
 * an entry on the device with more rows than any of its is reported
 * (TF_DEV_BAD_SEG) and skipped, here and in tf_kv_read_q8.
 */
TFS_API tf_status tf_kv_append_q8(const void *k_rows, const void *v_rows, int32_t n_rows_total,
                                  const tf_q8_cache *cache_host, const int32_t *page_table, int32_t page_table_len,
                                  const tf_seg *segs, int32_t n_segs, const tf_seg *segs_host,
                                  const int32_t *page_table_host, uint32_t *status, tf_stream_t stream);

/*
 * The reverse: the last n_rows keys of every stream (all of them when n_rows =
 * n_keys) from an 8-bit cache into bf16 pages, for calls that read bf16 pages
 * (a prompt chunk over a cached prefix: tf_paged_attn_prompt).  Key j goes to
 * slot j % page_size of page dst_page_table[pt_base + j / page_size] of
 * k_pool, v_pool; q_row is not used.  Every value is exact in bf16; a row whose
 * scale byte is 255 becomes NaN.  Nothing else in the pools changes.
 *
 *  k_pool, v_pool  bf16 [n_pages_dst][n_kv_heads][page_size][head_dim], 16-byte
 *                  aligned (written)
 *  dst_page_table  int32 [page_table_len], laid out as page_table is
 *  dst_page_table_host  optional host copy, checked as page_table_host is
 *
 * A key whose page id is outside its pool, on either side, is skipped
 * (TF_ERR_BAD_PAGE / TF_DEV_BAD_PAGE).  Streams must not share the pages they
 * write.
 */
TFS_API tf_status tf_kv_read_q8(const tf_q8_cache *cache_host, const int32_t *page_table, int32_t page_table_len,
                                const tf_seg *segs, int32_t n_segs, const tf_seg *segs_host,
                                const int32_t *page_table_host, void *k_pool, void *v_pool, int32_t n_pages_dst,
                                const int32_t *dst_page_table, const int32_t *dst_page_table_host, uint32_t *status,
                                tf_stream_t stream);

/*
 * Attention of every stream's rows over an 8-bit cache, partials and merge in
 * one call: what tf_paged_attn_decode (or, with full != 0,
 * tf_paged_attn_block) and tf_attn_merge compute, with K and V the values the
 * codes stand for.  Scores, softmax statistics and sums are held in fp32; a
 * weight, times its value row's scale, enters the value product with 22 bits and
 * at least to 2^-32 of the largest such product of its partial.
 * The tensor cores truncate their sums: with more than 8 queries a kv-head a
 * partial of n keys may lose n 2^-27 of them (chosen splits have up to 8,192
 * keys, as far as n_splits_max allows).
 *
 *  scale       > 0
 *  split_keys  keys a partial covers: 0 lets the library choose (from the host
 *              table when one is given, else ceil(n_keys / n_splits_max)
 *              rounded up to the page size, stream by stream); else >= 16
 *  n_splits_max  the most partials a stream may take; it sizes the workspace
 *
 * The host table sizes the launch: its row counts and its longest stream's
 * partials.  A call that is captured and replayed over a changing device table
 * is given a host table with the most rows and keys the replays will see; a
 * replay whose stream asks for more partials reports TF_DEV_SPLITS, one whose
 * stream has more rows than the launch holds TF_DEV_BAD_SEG, and those of the
 * stream's rows that the launch holds are flagged.  Without one the launch is
 * sized for n_splits_max partials of every stream, and decode rows do not take
 * the kernel made for them: slower.
 *
 *  workspace   device scratch of at least tf_paged_attn_q8_workspace_bytes(...)
 *              bytes, 16-byte aligned; needs no initialisation
 *  out         f32 or bf16 (out_dtype TF_OUT_F32 / TF_OUT_BF16: the bf16 rows are
 *              the f32 ones, rounded once) [n_rows_total][n_q_heads][head_dim],
 *              16-byte aligned
 *  flags       u8 [n_rows_total][n_q_heads]: 1 where a visible score, value or
 *              the output is nonfinite, or the table's entry is bad; out is NaN there
 *
 * Only the rows the table names are written.  Rows of different streams must
 * not overlap.  A stream has up to 2^30 keys (more: TF_ERR_UNSUPPORTED /
 * TF_DEV_BAD_SEG).  Other arguments, shapes and errors: tf_paged_attn_decode.
 */
TFS_API tf_status tf_paged_attn_q8(const void *q, int32_t n_rows_total, int32_t n_q_heads,
                                   const tf_q8_cache *cache_host, const int32_t *page_table, int32_t page_table_len,
                                   const tf_seg *segs, int32_t n_segs, const tf_seg *segs_host,
                                   const int32_t *page_table_host, float scale, int32_t full, int32_t split_keys,
                                   int32_t n_splits_max, void *workspace, size_t workspace_bytes, void *out,
                                   int32_t out_dtype, uint8_t *flags, uint32_t *status, tf_stream_t stream);

/* Workspace bytes tf_paged_attn_q8 needs for these sizes (0 on bad sizes and past 2^60). */
TFS_API size_t tf_paged_attn_q8_workspace_bytes(int32_t n_rows_total, int32_t n_q_heads, int32_t head_dim,
                                                int32_t n_splits_max);

/*
 * Attention of streams that share long prefixes, each prefix read once for all
 * of its rows (a system prompt, a prompt-cache hit).  prefixes[p] is a tf_seg
 * that names a run of query rows [q_row, q_row + n_rows) and a prefix's n_keys
 * keys in their own pages; every one of those rows sees all of them.  segs[s]
 * holds a stream's own rows and keys, after the prefix, as for
 * tf_paged_attn_decode (row i sees the first n_keys - n_rows + i + 1).  A row's
 * output is attention over its prefix's keys and its own, which equals one
 * tf_paged_attn_decode over the two page lists put end to end.
 *
 *  prefixes    tf_seg [n_prefixes] (device); the entries' rows must not
 *              overlap; a row no entry names has no prefix; n_rows = 0 is
 *              ignored, otherwise n_keys >= 1
 *  prefixes_host, segs_host  optional host copies, validated
 *  scale       > 0
 *  split_keys  keys a partial covers: 0 lets the library choose for the
 *              prefixes and for the streams (captured calls: as for
 *              tf_paged_attn_q8); else >= 16, for both
 *  n_prefix_splits, n_splits_max  the most partials a prefix and a stream may
 *              take; they size the workspace
 *  workspace   at least tf_paged_attn_shared_workspace_bytes(...) bytes,
 *              16-byte aligned; needs no initialisation
 *  out, out_dtype, flags  as for tf_paged_attn_q8; only the rows segs names
 *              are written
 *
 * Chosen splits of prefixes, and of streams with more than 8 queries a kv-head,
 * have up to 8,192 keys, as far as the splits given allow: longer partials lose
 * bits as tf_paged_attn_q8's do.
 *
 * Streams and prefixes have up to 2^30 keys each.  Other arguments, shapes and
 * errors: tf_paged_attn_decode.
 */
TFS_API tf_status tf_paged_attn_shared(const void *q, int32_t n_rows_total, int32_t n_q_heads, const void *k_pool,
                                       const void *v_pool, int32_t n_pages, int32_t page_size, int32_t n_kv_heads,
                                       int32_t head_dim, const int32_t *page_table, int32_t page_table_len,
                                       const tf_seg *prefixes, int32_t n_prefixes, const tf_seg *prefixes_host,
                                       const tf_seg *segs, int32_t n_segs, const tf_seg *segs_host,
                                       const int32_t *page_table_host, float scale, int32_t split_keys,
                                       int32_t n_prefix_splits, int32_t n_splits_max, void *workspace,
                                       size_t workspace_bytes, void *out, int32_t out_dtype, uint8_t *flags,
                                       uint32_t *status, tf_stream_t stream);

/* Workspace bytes tf_paged_attn_shared needs for these sizes (0 on bad sizes and past 2^60). */
TFS_API size_t tf_paged_attn_shared_workspace_bytes(int32_t n_rows_total, int32_t n_q_heads, int32_t head_dim,
                                                    int32_t n_prefix_splits, int32_t n_splits_max);

/*
 * Log probabilities of given tokens, entropy and top alternatives of logit
 * rows in one pass: beside tf_argmax_rows, what a server returns with a token.
 * Row r's distribution is softmax(scale * x[r, 0 .. n_cols)), scale an inverse
 * temperature in [2^-64, 2^64].  A logit of -infinity is a masked column: probability
 * 0, never an alternative.  A row with a NaN, a +infinity or no unmasked
 * column is flagged: its outputs are NaN and its ids -1.
 *
 *  logits          f32 or bf16 (logits_dtype TF_OUT_F32 / TF_OUT_BF16) [n_rows][ld],
 *                  aligned to its elements (16-byte rows are read faster)
 *  tokens          int32 [n_rows][n_tokens], n_tokens >= 0; a token outside
 *                  [0, n_cols) gives NaN and sets TF_DEV_BAD_TOKEN
 *  token_logprobs  f32 [n_rows][n_tokens]: log p of each given token (-infinity
 *                  for a masked one)
 *  entropy         f32 [n_rows], nullable: -sum p log p, in nats
 *  lse             f32 [n_rows], nullable: log sum exp(scale * x)
 *  top_k           alternatives a row, 0 to 32 (0: top_ids, top_logprobs may be null)
 *  top_ids         int32 [n_rows][top_k]: the columns of the largest logits, largest
 *                  first, ties to the lower id (-0 equals +0); -1 past the unmasked columns
 *  top_logprobs    f32 [n_rows][top_k]: their log p; -infinity past the unmasked columns
 *  flags           u8 [n_rows]
 *  status          uint32 device word for TF_DEV_BAD_TOKEN
 *
 * Supported: 1 <= n_cols <= 2^24, n_rows up to 2^31 - 1.
 */
TFS_API tf_status tf_logprob_rows(const void *logits, int32_t logits_dtype, int32_t n_rows, int32_t n_cols,
                                  int64_t ld, float scale, const int32_t *tokens, int32_t n_tokens,
                                  float *token_logprobs, float *entropy, float *lse, int32_t top_k, int32_t *top_ids,
                                  float *top_logprobs, uint8_t *flags, uint32_t *status, tf_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TFSERVE_H */
