/*
 * mxq_pages.h -- C ABI of libmxq, third part: serving from a packed KV cache
 * that is held in pages.  New rows quantized into their places, attention of
 * new tokens (one, or a tree of drafted ones) over the packed rows, and what a
 * serving loop does to pages: forking, freeing, reserving, compacting, and
 * moving a verified path of drafted rows together.
 *
 * The conventions of mxq.h hold here: device pointers owned by the caller, no
 * allocation, no synchronization, host-side checks that return a negative
 * mxq_status before any HIP call, MXQ_OK without a launch for empty problems,
 * dense row-major tensors.  int32 and float arrays are 4-byte aligned, pools
 * and q 16-byte (MXQ_ERR_ALIGN otherwise).  Every result is deterministic.
 *
 * Words used below
 * ----------------
 *  pool   the codes or the scale bytes of all pages: codes uint8 [pages,
 *         kv_heads, page_size, head_dim] (fp8) or [.., head_dim / 2] (mxfp4,
 *         nvfp4), scales uint8 [pages, kv_heads, page_size, head_dim / block],
 *         each row in the form of quantize_cache_packed.  A cache has such a
 *         pair for the keys and one for the values, or (v_codes and v_scales
 *         NULL) one for both: the values are the keys.
 *  table  int32 [sequences, width]: position p of a sequence lies in row
 *         p % page_size of page table[sequence][p / page_size].  An entry
 *         outside [0, pages) (-1) is no page: positions there do not exist,
 *         nothing is read or written for them.
 *  lengths int32 [sequences]: a sequence's cached positions.  Values below 0
 *         count as 0, values past width * page_size as that.
 *  refs   int32 [pages]: how many table entries name the page; a page with 0
 *         (or less) is free.
 * The rows of free pages, and those of positions that are neither cached nor
 * drafted, may hold anything.
 */
#ifndef MXQ_PAGES_H
#define MXQ_PAGES_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int64_t pages;      /* 1 .. 2^31 - 1 */
  int64_t page_size;  /* 16, 32, 64, 128 or 256 positions */
  int64_t kv_heads;   /* 1 .. 1024 */
  int64_t head_dim;   /* 64, 128, 256 or 512 */
  int32_t fmt;        /* mxq_format */
  int32_t block;      /* channels that share a scale: 16, 32, 64 or 128, no more than head_dim */
  uint8_t* k_codes;
  uint8_t* k_scales;
  uint8_t* v_codes;   /* both NULL: the values are the keys */
  uint8_t* v_scales;
} mxq_cache;

/*
 * cache_append -- rows k, v [sequences, tokens, kv_heads, head_dim] of dtype t
 * into the cache: row j of a sequence goes to position lengths + j, for
 * j < counts (int32 [sequences], NULL = tokens).  Codes and scale bytes are
 * those of quantize_cache_packed, bit for bit.  A row whose position has no
 * page, or a page that not exactly one table entry names (refs != 1), is not
 * written: what other sequences read stays as it is.  lengths does not change.
 * v is NULL if the cache has no pools of its own for the values.
 * Values must be finite.
 * Errors: MXQ_ERR_SHAPE (a size outside the ranges of mxq_cache, negative or
 * too large: sequences 2^20, tokens 2^20, width * page_size 2^30, 2^36 rows),
 * MXQ_ERR_DTYPE, MXQ_ERR_FORMAT, MXQ_ERR_BLOCK, MXQ_ERR_NULL, MXQ_ERR_ALIGN,
 * MXQ_ERR_ALIAS (a pool overlaps another buffer), MXQ_ERR_HIP.
 */
int cache_append(const mxq_cache* cache, const int32_t* table, int64_t sequences, int64_t width,
                 const int32_t* lengths, const int32_t* refs, const void* k, const void* v, int t, int64_t tokens,
                 const int32_t* counts, void* stream);

/*
 * cache_attention -- attention of new tokens over the cache.  q [sequences,
 * tokens, heads, head_dim] of dtype t; heads is a multiple of kv_heads, and
 * head h reads kv head h / (heads / kv_heads).  The new tokens' own keys and
 * values are in the cache already (cache_append): token j's at position
 * lengths + j.  Token i attends to
 *   every cached position (those below lengths), and
 *   position lengths + j for each j < counts that it may see: mask[i, j] != 0
 *   (uint8 [tokens, tokens], or with mask_each [sequences, tokens, tokens]:
 *   the tree; whatever it says, j may be after i), or j <= i where mask is NULL.
 * With s_p = scale * q . k_p over those positions,
 *   out = sum_p exp(s_p - m) v_p / sum_p exp(s_p - m), lse = m + log(sum_p
 *   exp(s_p - m)), m = max s_p.
 * out is [sequences, tokens, heads, head_dim] of dtype t, lse fp32 [sequences,
 * tokens, heads] (NULL: not wanted).  A token with nothing to attend to, and
 * tokens from counts on (int32 [sequences], NULL = tokens), get out = 0 and
 * lse = -inf.  Positions a token does not attend to may hold anything, NaN
 * too.  A value of 2^128 or more by size (code times scale) counts as an
 * infinity: a token that attends to it, however small the probability, gets
 * that infinity in its channel, or NaN where it attends to both signs or to a
 * NaN.  Keys that are attended to must be finite.  Keys, values and q enter the products as they are (q in as many bf16
 * parts as its type takes, or fp16), probabilities in enough bf16 or fp16 parts
 * that what is lost stays below the output's rounding; sums are fp32, of
 * probabilities that may be 2^8 times the largest (so that n values of 2^120 / n
 * or more by size may come out infinite).
 * workspace: cache_attention_workspace(the same sizes) bytes, 16-byte aligned;
 * its contents before and after the call mean nothing, and calls that may run
 * at the same time need one each.
 * Errors: as cache_append, and MXQ_ERR_SHAPE (heads not a multiple of
 * kv_heads or more than 2^14, tokens > 1024, more than 2^31 - 1 rows of q, a
 * scale of 2^127 or more by size or NaN, a workspace that is too small).  cache_attention_workspace returns
 * MXQ_ERR_SHAPE, MXQ_ERR_DTYPE, MXQ_ERR_FORMAT or MXQ_ERR_BLOCK for sizes that
 * cache_attention refuses; it reads no pool, whose pointers may be NULL.
 */
int64_t cache_attention_workspace(const mxq_cache* cache, int64_t sequences, int64_t width, int t, int64_t tokens,
                                  int64_t heads);
int cache_attention(const mxq_cache* cache, const int32_t* table, int64_t sequences, int64_t width,
                    const int32_t* lengths, const void* q, int t, int64_t tokens, int64_t heads, const uint8_t* mask,
                    int mask_each, const int32_t* counts, double scale, void* out, float* lse, void* workspace,
                    int64_t workspace_bytes, void* stream);

/*
 * cache_fork -- the table rows of `children` sequences, each continuing one of
 * the `sequences` given: table_out[c] = table[parents[c]] (parents int32
 * [children]; NULL: child c continues sequence c, children = sequences), and
 * lengths_out[c] = lengths[parents[c]].  A parent outside [0, sequences) gives
 * an empty sequence (no page, length 0).  With keep (int32 [children])
 * lengths_out is cut to keep (at least 0), and entries past the pages that the
 * remaining positions need become -1.  refs_out counts the new entries too, and
 * with release no longer the old ones.  No page is copied: cache_reserve gives
 * a sequence a page of its own before it is written to.
 * Outputs: table_out int32 [children, width], lengths_out int32 [children],
 * refs_out int32 [pages].  Out-of-range entries come out as -1.
 * Errors: MXQ_ERR_SHAPE (sequences or children negative or past 2^20, width not
 * in 1 .. 2^20, entries past 2^30, page_size, pages), MXQ_ERR_NULL,
 * MXQ_ERR_ALIGN, MXQ_ERR_ALIAS (outputs overlap anything), MXQ_ERR_HIP.
 */
int cache_fork(const int32_t* table, int64_t sequences, int64_t width, const int32_t* lengths, const int32_t* refs,
               int64_t pages, int64_t page_size, const int32_t* parents, int64_t children, const int32_t* keep,
               int release, int32_t* table_out, int32_t* lengths_out, int32_t* refs_out, void* stream);

/*
 * cache_reserve -- pages for the next tokens of every sequence (tokens, or
 * tokens_each int32 [sequences] where that is not NULL; below 0 counts as 0),
 * so that cache_append can write positions lengths .. lengths + tokens - 1.
 * Each entry of these positions that has no page, or a page that other entries
 * name too (refs > 1), gets a free one.  Of a page that others name, the rows
 * below lengths (the first entry's, where lengths % page_size > 0) are copied;
 * rows behind them are not.  If all entries that name a page ask for it in one
 * call, the last of them keeps it.
 * Free pages are taken in rising order, sequence by sequence, entry by entry.
 * short_out int32 [sequences] says how many pages a sequence lacks in the end:
 * the pool ran out, its row of the table is too short, or a page could not be
 * made its own.  Where it is 0, every entry of the positions names a page with
 * refs_out 1.
 * Outputs: table_out, refs_out like table and refs; copied rows in the pools.
 * workspace: cache_reserve_workspace(sequences, width, pages) bytes, 4-byte
 * aligned, as for cache_attention.
 * Errors: as cache_append, and MXQ_ERR_SHAPE (more than 4096 sequences, tokens
 * past 2^30, a workspace that is too small).
 */
int64_t cache_reserve_workspace(int64_t sequences, int64_t width, int64_t pages);
int cache_reserve(const mxq_cache* cache, const int32_t* table, int64_t sequences, int64_t width,
                  const int32_t* lengths, const int32_t* refs, int64_t tokens, const int32_t* tokens_each,
                  int32_t* table_out, int32_t* refs_out, int32_t* short_out, void* workspace, int64_t workspace_bytes,
                  void* stream);

/*
 * cache_accept -- the rows of accepted drafted tokens moved together: row
 * lengths + accepted[a] to position lengths + a, lengths_out = lengths + the
 * count.  accepted int32 [sequences, most], most <= 64: draft numbers in rising
 * order; a sequence's list ends before the first value that is negative or no
 * larger than the one before it, or whose position or place has no page, or
 * whose place lies in a page that not exactly one entry names.
 * Errors: as cache_append, and MXQ_ERR_SHAPE (most > 64).
 */
int cache_accept(const mxq_cache* cache, const int32_t* table, int64_t sequences, int64_t width,
                 const int32_t* lengths, const int32_t* refs, const int32_t* accepted, int64_t most,
                 int32_t* lengths_out, void* stream);

/*
 * cache_compact -- the pages in use moved to the front of the pool: of n used
 * pages (refs > 0) those with an index of n or more are copied, in rising
 * order, to the free ones below n.  table_out and refs_out follow.  The table
 * must hold every entry that names a page.
 * workspace: cache_compact_workspace(pages) bytes, 4-byte aligned, as above.
 * Errors: as cache_append, and MXQ_ERR_SHAPE (a workspace that is too small).
 */
int64_t cache_compact_workspace(int64_t pages);
int cache_compact(const mxq_cache* cache, const int32_t* table, int64_t sequences, int64_t width, const int32_t* refs,
                  int32_t* table_out, int32_t* refs_out, void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_PAGES_H */
