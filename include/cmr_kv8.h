/*
 * cmr_kv8.h -- a paged KV cache held in 8 bits, as a C ABI over hand-written
 * sm_100a (B200) CUDA kernels: the M-RoPE rotation that writes it, the
 * attention that reads it, and the upkeep of its pages.
 *
 * The cache.  Tokens live in pages of page_tokens (P) each, 16, 32, 64 or 128:
 *   k_pages, v_pages    uint8 (e4m3) [num_layers, num_pages, hk, P, head_dim]
 *   k_scales, v_scales  float [num_layers, num_pages, hk]
 * A value is its code times its page's scale.  Scales are powers of two
 * between 2^-60 and 2^60 (cmr_kv8_rotate_qk writes only those), so a page whose
 * scale has to grow re-encodes the codes it holds by changing exponents: a
 * code loses bits only where it falls below e4m3's smallest normal number.
 * A finite value beyond 448 * 2^60 is held as +-448 * 2^60; an infinity or a
 * NaN is held as NaN (code 0x7f) and does not enter the scale.
 *   page_table          int32 [table_rows, max_pages]: row r lists the pages of
 *                       one sequence in order, -1 behind the last; the token
 *                       at absolute index p is row p % P of page
 *                       page_table[r][p / P] (the same page id in every layer)
 *   page_refs           int32 [num_pages]: how many rows of the table hold the
 *                       page, 0 for a free page
 * Sequence b of a call uses table row slot[b], or row b where slot is NULL.
 *
 * Conventions (pointers, streams, errors, device status word, no allocation
 * and no synchronisation in the library, no traps, bounded waits) are those of
 * cmr.h.  cmr_kv8_last_error_message() has the reason for the last failure.
 */
#ifndef CMR_KV8_H_
#define CMR_KV8_H_

#include "cmr.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further bits of the optional device status word. */
#define CMR_DEVICE_PAGES_FULL 8  /* no free page was left: see the call's own words */
#define CMR_DEVICE_BAD_SCALE 16  /* a scale that is not within 2^-60 .. 2^60 */

/* Rotate Q in place and write the rotated K rows and the V rows of a batch of
 * tokens into the 8-bit cache: cmr_rotate_qk_cache with this cache in the place
 * of its bf16 one.  Token t of sequence b (cu[b] <= t < cu[b+1]) sits at
 * absolute index p = pos_offset[b] + t - cu[b] and gets the canvas planes of p
 * under (start[b], amount[b]).  What is encoded is the rotated K as
 * cmr_rotate_qk_cache would store it, in bf16, and V as given.
 * A page whose row 0 is written by the call gets the smallest power of two s with
 * max |value written| <= 448 s; the rows behind those written are left as they
 * are.  A page that held rows before (pos_offset[b] % P of them) keeps its scale
 * unless the new rows need a larger one; then its earlier rows are re-encoded.
 * Rows behind the last sequence (t >= cu[num_seqs]) are left as they are, in Q
 * too.
 *
 *   q                 device bf16 [num_layers, n_tokens, hq, head_dim], in place
 *   k, v              device bf16 [num_layers, n_tokens, hk, head_dim], read only
 *   cu_seqlens        device int32 [num_seqs + 1], cu[0] = 0, non-decreasing, at
 *                     most n_tokens; or NULL when num_seqs == n_tokens and
 *                     each sequence holds one token (a decode step)
 *   pos_offset        device int32 [num_seqs], or NULL for all zeros
 *   start, amount     device int32 [num_seqs], as cmr_positions gives them
 *   head_dim          64, 128 or 256
 *   theta, sections, rot_dim   as in cmr_rotate_qk
 *   the cache, slot   as above; a page must not be written for two sequences in
 *                     one call, and one that several rows share must not be
 *                     written at all
 *   device_status     optional: CMR_DEVICE_CACHE_RANGE where a token's index,
 *                     table row or page lies outside the cache (its K and V are
 *                     then not written; Q is rotated), CMR_DEVICE_BAD_SCALE where
 *                     a page held rows under such a scale (they are left as they
 *                     are, and the page gets the new rows' scale),
 *                     CMR_DEVICE_BAD_CU_SEQLENS (the sequences involved
 *                     are skipped)
 * hq may be 0 (q NULL); hk >= 1.  q, k, v, k_pages and v_pages 16-byte aligned; q must
 * not overlap k or v, nor any of them the pages.
 * Errors: CMR_EINVAL for any violation above, CMR_EUNSUPPORTED for another
 * head_dim or page_tokens, hk * head_dim over 2^23, hk * num_layers over 65535, or
 * num_layers * num_pages * hk or (hq + hk) * num_layers over INT32_MAX. */
CMR_API cmr_status cmr_kv8_rotate_qk(void* q, const void* k, const void* v,
                                     const int32_t* cu_seqlens, int32_t num_seqs,
                                     const int32_t* pos_offset, const int32_t* start,
                                     const int32_t* amount, int64_t n_tokens, int32_t num_layers,
                                     int32_t hq, int32_t hk, int32_t head_dim, double theta,
                                     const int32_t sections[3], int32_t rot_dim, void* k_pages,
                                     void* v_pages, float* k_scales, float* v_scales,
                                     int32_t num_pages, int32_t page_tokens,
                                     const int32_t* page_table, int32_t table_rows,
                                     int32_t max_pages, const int32_t* slot,
                                     int32_t* device_status, cmr_stream_t stream);

/* Causal attention over the cache.  Query token t of sequence b sits at absolute
 * index p = pos_offset[b] + t - cu[b] and sees the sequence's indices 0 .. p (its
 * own key and value are in the cache already):
 *   out[l, t, h, :] = sum_i w_i v_i / sum_i w_i,  w_i = exp(scale * q[l, t, h, :] . k_i)
 * with k_i, v_i of KV head h / (hq / hk).  The sums and the softmax run in fp32;
 * for the product with the codes of the values the weights, times their page's value
 * scale, are rounded: in the kernel for few rows (below) by at most 2^-11 of themselves,
 * or 2^-38 of the row's largest where that is more; in the one for many by 2^-9 + 2^-11,
 * or 2^-26.  The result is rounded to bf16.  A token with p < 0 sees nothing and gets zeros.
 * Rows behind the last sequence are left as they are.
 * Rows of the pages that a token does not see never reach its result, whatever
 * their codes are (NaN among them).
 *
 *   q, out            device bf16 [num_layers, n_tokens, hq, head_dim], 16-byte
 *                     aligned; out must not overlap q or the cache
 *   hq                a positive multiple of hk, hq / hk <= 128
 *   scale             finite; the softmax scale (1 / sqrt(head_dim) in this model)
 *   workspace         device memory, 16-byte aligned, of at least
 *                     cmr_kv8_attend_workspace_bytes; its contents before and
 *                     after a call do not matter, but calls that can overlap on
 *                     the device must not share it (a captured graph keeps its own)
 *   device_status     optional: CMR_DEVICE_CACHE_RANGE where a token sees an
 *                     index that lies outside the cache, CMR_DEVICE_BAD_SCALE where
 *                     it sees a page with such a scale (in both cases it is as if
 *                     those indices were not there), CMR_DEVICE_BAD_CU_SEQLENS,
 *                     CMR_DEVICE_WAIT_TIMEOUT
 *   the rest          as in cmr_kv8_rotate_qk
 * Scores (scale * q . k) have to lie within fp32's range.
 * One kernel shares each key and value among 8 or 16 query rows (tokens x hq / hk) and
 * is bound by reading the cache, another takes 128 rows on the tensor cores.  A decode
 * step runs the first for hq / hk up to 16.  With cu_seqlens, whose lengths only the
 * device knows, a call of more than 64 rows runs the second when there are more than
 * 8 rows per sequence on average, and otherwise both, the second for the sequences
 * of more than 32 rows.
 * Errors: as cmr_kv8_rotate_qk, and CMR_EINVAL when max_pages * page_tokens is over
 * INT32_MAX - 256. */
CMR_API cmr_status cmr_kv8_attend(const void* q, void* out, const int32_t* cu_seqlens,
                                  int32_t num_seqs, const int32_t* pos_offset, int64_t n_tokens,
                                  int32_t num_layers, int32_t hq, int32_t hk, int32_t head_dim,
                                  double scale, const void* k_pages, const void* v_pages,
                                  const float* k_scales, const float* v_scales,
                                  int32_t num_pages, int32_t page_tokens,
                                  const int32_t* page_table, int32_t table_rows,
                                  int32_t max_pages, const int32_t* slot, void* workspace,
                                  size_t workspace_bytes, int32_t* device_status,
                                  cmr_stream_t stream);

/* Workspace bytes of cmr_kv8_attend for these sizes (0 for sizes that it refuses
 * or that leave nothing to do).  The count of SMs of the current device enters. */
CMR_API size_t cmr_kv8_attend_workspace_bytes(int32_t num_seqs, int64_t n_tokens,
                                              int32_t num_layers, int32_t hq, int32_t hk,
                                              int32_t head_dim);

/* ---- pages.  The table and the counts are the state; it lives on the device and
 * these calls change it there, in stream order, without the host's help.  Free
 * pages are given out lowest index first, to the entries of a call in order, so
 * the same calls always give the same table.
 *
 *   slots (src, dst)  device int32 [n]: rows of the table.  An entry outside the
 *                     table, or one named earlier in the same call (dst of a
 *                     fork), is skipped with CMR_DEVICE_CACHE_RANGE
 *   lens              device int32 [n]: tokens
 *   workspace         device memory, 16-byte aligned, of at least
 *                     cmr_kv8_pages_workspace_bytes(table_rows, num_pages, n); as
 *                     for cmr_kv8_attend, overlapping calls need their own
 * A row's entries up to the first negative one are its pages, whatever stands behind
 * it; a page id outside the pool in them sets CMR_DEVICE_CACHE_RANGE and is not
 * followed (a fork looks at those that it shares or copies from). */

/* Give each named row the pages that it lacks to hold lens[i] tokens (none where
 * it has them).  An entry that needs more than max_pages gets none
 * (CMR_DEVICE_CACHE_RANGE); one that finds too few free pages left, and those behind
 * it that need any, get none (CMR_DEVICE_PAGES_FULL).
 * New pages get page_refs = 1; their codes and scales are left as they are.  A page id
 * outside the pool counts as a page of its row. */
CMR_API cmr_status cmr_kv8_extend(int32_t* page_table, int32_t table_rows, int32_t max_pages,
                                  int32_t* page_refs, int32_t num_pages, int32_t page_tokens,
                                  const int32_t* slots, const int32_t* lens, int32_t n,
                                  void* workspace, size_t workspace_bytes,
                                  int32_t* device_status, cmr_stream_t stream);

/* Make row dst[i], which must be empty, a second holder of the first lens[i] tokens
 * of row src[i]: the whole pages are shared (page_refs + 1), and where lens[i] does
 * not end with a page the rest of its tokens are copied, in every layer, with
 * the page's scales, into a page of dst[i]'s own, so that both can be written on.
 * An entry whose src has fewer pages than lens[i] needs, whose dst is not empty or
 * whose lens[i] is negative is skipped with CMR_DEVICE_CACHE_RANGE; one that finds
 * no free page, with CMR_DEVICE_PAGES_FULL.  All rows are read as they were before
 * the call. */
CMR_API cmr_status cmr_kv8_fork(void* k_pages, void* v_pages, float* k_scales, float* v_scales,
                                int32_t num_layers, int32_t hk, int32_t head_dim,
                                int32_t num_pages, int32_t page_tokens, int32_t* page_table,
                                int32_t table_rows, int32_t max_pages, int32_t* page_refs,
                                const int32_t* src, const int32_t* dst, const int32_t* lens,
                                int32_t n, void* workspace, size_t workspace_bytes,
                                int32_t* device_status, cmr_stream_t stream);

/* Empty the named rows: page_refs - 1 for each of their pages (a page at 0 is free;
 * one that is at 0 already sets CMR_DEVICE_CACHE_RANGE and stays there), and -1 in
 * the entries that held them. */
CMR_API cmr_status cmr_kv8_free(int32_t* page_table, int32_t table_rows, int32_t max_pages,
                                int32_t* page_refs, int32_t num_pages, const int32_t* slots,
                                int32_t n, int32_t* device_status, cmr_stream_t stream);

/* Move pages so that those in use are the pool's first: with c pages in use, the
 * ones at c and above go, in order, to the free ones below c, in every layer,
 * with their scales and counts, and the whole table follows.  page_refs > 0 says
 * that a page is in use.  Page ids held outside the table become stale.  Where a row
 * lists a page of c or above that is not in use, or one outside the pool, its entry is
 * left as it is (CMR_DEVICE_CACHE_RANGE). */
CMR_API cmr_status cmr_kv8_compact(void* k_pages, void* v_pages, float* k_scales,
                                   float* v_scales, int32_t num_layers, int32_t hk,
                                   int32_t head_dim, int32_t num_pages, int32_t page_tokens,
                                   int32_t* page_table, int32_t table_rows, int32_t max_pages,
                                   int32_t* page_refs, void* workspace, size_t workspace_bytes,
                                   int32_t* device_status, cmr_stream_t stream);

/* Workspace bytes of the calls above that take one (n = 0 for cmr_kv8_compact).  No CUDA
 * call is made. */
CMR_API size_t cmr_kv8_pages_workspace_bytes(int32_t table_rows, int32_t num_pages, int32_t n);

/* The calls above with their arguments in an array, one 8-byte word each, in order
 * and the stream among them (integers and addresses as int64, doubles as they are),
 * for bindings to which each argument is a cost of its own.
 *   call   0 cmr_kv8_rotate_qk (28 words), 1 cmr_kv8_attend (25), 2 cmr_kv8_extend (13),
 *          3 cmr_kv8_fork (21), 4 cmr_kv8_free (9), 5 cmr_kv8_compact (17)
 * With CMR_KV8_KNOWN_ADDRESSES added to its number a call does not look up where its
 * addresses lie, for bindings that know them to be memory of the current device.
 * Errors: those of the call, CMR_EINVAL for another number or count of words. */
#define CMR_KV8_KNOWN_ADDRESSES 256
CMR_API cmr_status cmr_kv8_call(int32_t call, const void* words, int32_t count);

/* Name of the kernel that the calling thread's last cmr_kv8_attend enqueued
 * ("attend_rows_kernel", "attend_tiles_kernel", or both with ", " between); "" before
 * the first. */
CMR_API const char* cmr_kv8_last_attend_kernel(void);

/* One-line reason for the last non-CMR_OK return of a cmr_kv8_ call on the calling
 * thread. */
CMR_API const char* cmr_kv8_last_error_message(void);

#ifdef __cplusplus
}
#endif

#endif /* CMR_KV8_H_ */
