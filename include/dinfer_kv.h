/*
 * dinfer_kv.h -- paged key/value cache: its pages, attention of one new token
 * per sequence over them, and prompt attention with a sliding window.
 *
 * The context of dinfer.h keeps every sequence's keys and values in one
 * contiguous slab.  A server that runs many sequences of different lengths
 * keeps them in pages instead: a sequence is a row of page numbers, pages are
 * handed out as it grows, and sequences that begin alike share pages.  These
 * entry points are that cache and the two attentions a serving loop needs
 * around it:
 *
 *   prompt:  dinfer_kv_extend, per layer { dinfer_op_window_attention over the
 *            prompt's own rows (dinfer_op_rope in front), dinfer_kv_append of its
 *            keys and values }
 *   token:   dinfer_kv_extend by one, per layer { dinfer_kv_append,
 *            dinfer_kv_attention }; with rotary positions dinfer_kv_append_rope,
 *            for sequences that begin alike dinfer_kv_prefix_attention
 *   between: dinfer_kv_fork, dinfer_kv_free, dinfer_kv_compact
 *
 * Conventions (those of dinfer_ops.h, and)
 *   - All pointers are device pointers unless stated; every call is
 *     asynchronous on `stream` (a cudaStream_t, NULL = legacy default stream),
 *     allocates nothing, and can be captured into a CUDA graph
 *     (dinfer_kv_status waits, and cannot).
 *   - The caller owns all memory, the cache's tables included.  Calls on one
 *     cache must be ordered on the GPU; only dinfer_kv_attention and
 *     dinfer_kv_prefix_attention calls may overlap with one another, each with
 *     a workspace of its own.
 *   - What the host cannot see (sequence numbers, page numbers, free pages) is
 *     checked on the device: the entry is skipped, and a bit is set in the
 *     cache's status word (dinfer_kv_status).  int32 operands (sequence numbers,
 *     row bounds, tables) are 4-byte aligned, or the call is refused.
 */
#ifndef DINFER_KV_H
#define DINFER_KV_H

#include "dinfer_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The cache.  Element (layer l, page p, slot t, head h, i) of k and of v lies
 * at l * layer_stride + p * page_stride + t * token_stride + h * head_stride
 * + i elements; any order of these dimensions that does not overlap will do.
 * k, v: 16-byte aligned, all strides multiples of 16 bytes.  dtype DINFER_BF16
 * or DINFER_FP32, head_dim 64 or 128, page_size 1 .. 65536, kv_heads 1 .. 1024,
 * max_pages * page_size < 2^31, page_size * kv_heads * head_dim < 2^31.
 *   table [max_seqs][max_pages]  the pages of each sequence in order, -1 behind its last
 *   lens  [max_seqs]             tokens of each sequence (0: not in use); it holds ceil(len / page_size) pages
 *   refs  [num_pages]            how many sequences hold each page (0: free)
 *   state [dinfer_kv_state_ints] the library's: zero it before the first call and
 *                                whenever table, lens or refs are written by hand (not by dinfer_kv_set)
 * An empty cache is table all -1, the others all 0. */
typedef struct dinfer_kv_cache {
  void* k;
  void* v;
  int64_t layer_stride, page_stride, token_stride, head_stride;
  int32_t* table;
  int32_t* lens;
  int32_t* refs;
  int32_t* state;
  int32_t n_layers, num_pages, page_size, kv_heads, head_dim, dtype;
  int32_t max_seqs, max_pages;
} dinfer_kv_cache;

/* int32 elements of `state` (host-side arithmetic; 0 for bad sizes). */
size_t dinfer_kv_state_ints(int32_t num_pages, int32_t max_seqs);

/* Bits of the status word. */
enum {
  DINFER_KV_BAD_SEQ = 1,  /* a sequence number out of range, named twice where once is allowed, a fork onto one in use */
  DINFER_KV_NO_PAGES = 2, /* not enough free pages */
  DINFER_KV_BAD_PAGE = 4, /* a table entry inside a sequence's length is no page of the cache */
  DINFER_KV_SHARED = 8,   /* rows appended to a page that other sequences hold too */
  DINFER_KV_FULL = 16     /* a sequence beyond max_pages pages; more rows than tokens, or row bounds out of order or
                             behind k's last row */
};

/* Waits for `stream`, reads the status word into *bits (host, may be NULL)
 * and clears it.  DINFER_EDEVICE if any bit was set (dinfer_last_error names
 * them), else DINFER_OK. */
dinfer_status dinfer_kv_status(const dinfer_kv_cache* cache, uint32_t* bits, void* stream);

/* Takes over another set of tables of the cache's sizes (a snapshot, a plan
 * made elsewhere), and clears the state and its status. */
dinfer_status dinfer_kv_set(const dinfer_kv_cache* cache, const int32_t* table, const int32_t* lens,
                            const int32_t* refs, void* stream);

/* Sequence seqs[i] (NULL: i) grows by add[i] >= 0 tokens (NULL: one each):
 * its len rises and the pages this takes are handed out, lowest free page
 * first, entries in order.  When the free pages run out, the entry they no
 * longer suffice for and every later one that needs pages stay as they were
 * (DINFER_KV_NO_PAGES).  A sequence named twice grows by its first entry
 * (DINFER_KV_BAD_SEQ).  1 <= n <= 1024.  The new tokens' slots hold whatever
 * the pages held until dinfer_kv_append writes them. */
dinfer_status dinfer_kv_extend(const dinfer_kv_cache* cache, const int32_t* seqs, const int32_t* add, int32_t n,
                               void* stream);

/* Keys and values of the last rows of each sequence in one layer: rows
 * rows[i] .. rows[i + 1] - 1 of k and v (NULL: row i alone) are the last ones
 * of sequence seqs[i] (NULL: i), whose len already counts them.
 * k, v [total_rows][kv_heads][head_dim], head rows packed, consecutive rows
 * k_stride / v_stride elements apart (multiples of 16 bytes; slices of one
 * projection's output will do), in the cache's type, 16-byte aligned.  rows
 * [n + 1] is non-decreasing, from 0 or more to at most total_rows (else
 * DINFER_KV_FULL); rows of k before rows[0] or behind rows[n] are not stored.  Rows
 * that fall on a page other sequences hold are not stored (DINFER_KV_SHARED).
 * A sequence named twice takes its first entry's (DINFER_KV_BAD_SEQ).
 * 1 <= n <= 1024, without seqs n <= max_seqs. */
dinfer_status dinfer_kv_append(const dinfer_kv_cache* cache, int32_t layer, const int32_t* seqs, const int32_t* rows,
                               int32_t n, const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                               int32_t total_rows, void* stream);

/* dinfer_kv_append whose keys are rotated on the way, each at its token's place in
 * its sequence, or at positions[row] where positions [total_rows] is given.  q
 * (optional, NULL with q_out): [total_rows][heads][head_dim], the rows' queries, go
 * rotated alike to q_out, which is q, with the same stride, or overlaps no operand.  q,
 * q_out: head rows packed, rows q_stride / q_out_stride elements apart, 1 <= heads <=
 * 65536, in the cache's type and alignment.  A row that is not stored (see
 * dinfer_kv_append) leaves its row of q_out as it was.  rope as in dinfer_op_rope. */
dinfer_status dinfer_kv_append_rope(const dinfer_kv_cache* cache, int32_t layer, const dinfer_rope* rope,
                                    const int32_t* positions, const int32_t* seqs, const int32_t* rows, int32_t n,
                                    const void* q, void* q_out, int32_t heads, int64_t q_stride, int64_t q_out_stride,
                                    const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                                    int32_t total_rows, void* stream);

/* Sequence dst[i], which must not be in use, becomes a copy of sequence
 * src[i].  share != 0: the full pages are held by both, the partly filled last
 * one is copied in every layer.  share == 0: every page is copied (for
 * sequences whose slots are rewritten, as block decoding does).  Copies take
 * the tokens alone; the other slots of a new page stay as they were.  Pages
 * are handed out as in dinfer_kv_extend.  One src may be forked many times;
 * a dst named twice takes its first entry.  All src are copied as they were
 * before the call: a src that is also a dst of the same call is still empty,
 * and its copy too (chains of forks take a call each).  1 <= n <= 1024. */
dinfer_status dinfer_kv_fork(const dinfer_kv_cache* cache, const int32_t* src, const int32_t* dst, int32_t n,
                             int32_t share, void* stream);

/* Sequences seqs[0 .. n - 1] let go of their pages; len becomes 0, the table
 * row -1.  Sequences not in use stay so. */
dinfer_status dinfer_kv_free(const dinfer_kv_cache* cache, const int32_t* seqs, int32_t n, void* stream);

/* Packs the pages in use to the front: with c of them in use, the j-th free
 * page below c takes the j-th used page at or above c, in every layer, and the
 * tables follow.  live (optional, int32) receives c. */
dinfer_status dinfer_kv_compact(const dinfer_kv_cache* cache, int32_t* live, void* stream);

/* Attention of each sequence's last token over its pages in one layer:
 *   o[i, h, :] = sum_j softmax_j(scale * q[i, h, :] . K[j, h', :]) V[j, h', :]
 * over the keys j < len of sequence seqs[i] (NULL: i) with
 *   window < 0 (all), or j >= len - 1 - window, or j < sinks,
 * h' = h / (heads / kv_heads).  q, o [n][heads][head_dim] in the cache's type,
 * head rows packed, rows q_stride / o_stride elements apart, 16-byte aligned.
 * A sequence without tokens, or whose scores are all -inf, gives zeros.  Keys
 * on a table entry that is no page are left out (DINFER_KV_BAD_PAGE).
 * A sequence may be named more than once, and o may be q.  heads % kv_heads == 0,
 * heads <= 65536, 1 <= n <= 1024, scale > 0.  The host knows no lengths, so it
 * refuses calls whose sequences could add up to 2^31 steps of keys: none with
 *   n * heads * (keys / 16 + 11) < 2^31,
 * keys = max_pages * page_size or, with a window, window + 1 + sinks if that is
 * less.  The keys are split over the GPU and joined in a
 * fixed order: the same call gives the same bits. */
dinfer_status dinfer_kv_attention(const dinfer_kv_cache* cache, int32_t layer, const int32_t* seqs, int32_t n,
                                  const void* q, void* o, int64_t q_stride, int64_t o_stride, int32_t heads,
                                  int32_t window, int32_t sinks, float scale, void* workspace, size_t workspace_bytes,
                                  void* stream);

/* dinfer_kv_attention (all keys) where groups of entries begin alike: entries
 * groups[g] .. groups[g + 1] - 1 (groups NULL with n_groups 1: all) hold the same pages
 * for their first prefix[g] tokens, as dinfer_kv_fork with share leaves them; those keys
 * and values are read once for the whole group.  Of prefix[g] the whole pages count that
 * every sequence of the group with tokens has beyond its last token's own; 0 or less, or a
 * group with a single such sequence, shares nothing.  The pages read are those of the
 * group's first sequence with tokens; another that does not hold them sets
 * DINFER_KV_BAD_SEQ.  Entries of no group are computed by themselves; where bounds
 * are out of order or beyond n no group shares anything (DINFER_KV_FULL).  groups [n_groups + 1], prefix [n_groups],
 * 1 <= n_groups, n + n_groups <= 1024; everything else as in dinfer_kv_attention, but that
 * the sums of all rows have to fit the workspace:
 *   n * heads * (16 * head_dim + 32) bytes beside 32 MiB, and
 *   (2 n + n_groups) * heads * (max_pages * page_size / 16 + 11) < 2^31. */
dinfer_status dinfer_kv_prefix_attention(const dinfer_kv_cache* cache, int32_t layer, const int32_t* seqs, int32_t n,
                                         const int32_t* groups, const int32_t* prefix, int32_t n_groups, const void* q,
                                         void* o, int64_t q_stride, int64_t o_stride, int32_t heads, float scale,
                                         void* workspace, size_t workspace_bytes, void* stream);

/* Attention of many rows with a sliding window and sinks, over `batch` ragged
 * sequences:  sequence b has the query rows cu_q[b] .. cu_q[b + 1] - 1 and the
 * key rows cu_k[b] .. cu_k[b + 1] - 1; its row i stands at position
 * p = (keys - rows) + i and sees key j if
 *   (right < 0 or j <= p + right) and (left < 0 or j >= p - left or j < sinks).
 * left = -1, right = 0 is causal, -1, -1 sees everything (the block decoder's
 * attention), both >= 0 a vicinity.  A row that sees no key, or whose scores are
 * all -inf, gives zeros.
 * q, o [total_q][heads][head_dim], k, v [total_k][kv_heads][head_dim], dtype
 * DINFER_BF16 or DINFER_FP32, head rows packed, rows x_stride elements apart
 * (multiples of 16 bytes), 16-byte aligned.  cu_q, cu_k: int32 [batch + 1],
 * non-decreasing, or both NULL with batch 1 (all rows).  Rows of o outside
 * every sequence stay as they were.  1 <= batch <= 1024, 1 <= total_q, total_k
 * <= 2^30, head_dim 64 or 128, scale > 0; o must not overlap q, k or v.
 * bf16 runs on the tensor cores: probabilities are rounded to bf16 and summed
 * in fp32.  fp32 is computed in fp32.  Keys that a row does not see do not
 * touch it, whatever they hold.  The workspace may be NULL; when given, calls
 * that overlap need one each, a wait that timed out sets its status word (zero
 * it again then), and few rows over many keys are split over the keys and
 * joined in a fixed order: the same call gives the same bits. */
dinfer_status dinfer_op_window_attention(const void* q, const void* k, const void* v, void* o, int32_t dtype,
                                         int32_t batch, const int32_t* cu_q, const int32_t* cu_k, int32_t total_q,
                                         int32_t total_k, int32_t heads, int32_t kv_heads, int32_t head_dim,
                                         int64_t q_stride, int64_t k_stride, int64_t v_stride, int64_t o_stride,
                                         int32_t left, int32_t right, int32_t sinks, float scale, void* workspace,
                                         size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DINFER_KV_H */
