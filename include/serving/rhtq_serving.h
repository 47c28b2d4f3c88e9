/*
 * rhtq_serving.h -- what uses 4-bit rows when a model answers: products with quantised weights and a
 * paged 4-bit key-value cache (gfx950).
 *
 * The calls ship in librhtq.so beside those of rhtq.h and share their status codes, type codes and
 * conventions: device pointers owned by the caller, nothing allocated or kept, only kernels enqueued on
 * `stream` (so every call can be captured into a HIP graph), arguments checked on the host before any HIP
 * call.  Scratch memory is the caller's too; its contents need not be kept between calls and are
 * undefined afterwards.  Two calls that may run at the same time need workspaces of their own.
 *
 * Why rotated rows can be used as they lie: the rotation R = H diag(s) / sqrt(n) is orthonormal, so
 * q . k = (R q) . (R k), and sum_j p_j v_j = R^T sum_j p_j (R v_j).  A call rotates its few input rows once,
 * works on the codes, and undoes the rotation once on its output (QuaRot reviews page, review 2 Summary:
 * the rotation is invertible; review 3 Strengths: it is applied to activations and to the KV cache).
 */
#ifndef RHTQ_SERVING_H
#define RHTQ_SERVING_H

#include <stdint.h>

#include "../rhtq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define RHTQ_SERVING_VERSION 1
int rhtq_serving_version(void);

/*
 * Product with 4-bit weights:  y[t][r] = sum_k (R x[t])[k] * w_hat[r][k], where w_hat are the dequantised
 * rows of `packed` -- that is, y = x W^T with W the matrix rhtq_inverse would give for the same bytes.
 *   x          [tokens][n] bf16, fp16 or fp32; rotated != 0 says that it is R x already (signs, block unused)
 *   block      n for the plain rotation, or the block of a block-diagonal one (as rhtq_rotate_blocked)
 *   packed     [rows][n/2], scales [rows][n/group], tensor_scale (NVFP4) as rhtq_forward writes them for the
 *              weight's rows; group 0 = one INT4 scale per row
 *   y_out      [tokens][rows] in out_dtype (RHTQ_IN_BF16, RHTQ_IN_F16 or RHTQ_IN_F32)
 *   workspace  rhtq_matvec_workspace(...) bytes, 16-byte aligned
 * n: a multiple of 32 up to 2^20 (with rotated == 0 also one that rhtq_rotate or its blocked form takes).
 * rows up to 2^31 - 1024, tokens up to 2^20 (0: nothing to do).  Sums are in fp32; R x is carried to 22 bits, and to
 * 2^-35 of the largest value of its row.  A value of R x that is not finite gives NaN for its token.
 * packed must be 16-byte aligned, x, y_out and signs 16 bytes, scales to their element (NVFP4: 2 bytes).
 */
int64_t rhtq_matvec_workspace(int64_t tokens, int32_t n, int64_t rows);
int rhtq_matvec(const void* x, int in_dtype, int64_t tokens, int32_t n, int32_t block, const int8_t* signs,
                int rotated, const uint8_t* packed, const void* scales, const float* tensor_scale, int64_t rows,
                int fmt, int32_t group, int scale_dtype, void* y_out, int out_dtype, void* workspace,
                int64_t workspace_bytes, rhtq_stream_t stream);

/*
 * The cache.  One layer's keys (and, apart, its values) lie as
 *   codes   [pages][kv_heads][page][head_dim/2] bytes (16-byte aligned), scales [pages][kv_heads][page] fp32 or fp16 (aligned to their
 *           element, for attention to two, for page calls to 16 bytes),
 * each row an INT4 row of rhtq_forward with one scale (group = head_dim).  head_dim 64, 128 or 256; page a
 * power of two, 16 to 256.  Position p of a sequence lies in page table[seq][p / page], slot p % page;
 * `table` is [seqs][width] int32.  An entry outside [0, pages) is no page: its positions are not stored, read as
 * zero and seen by no query.  A length beyond width * page counts as width * page, a negative one as 0.
 * Limits: width * page below 2^31 - 256 and up to 2^31 - 2^23 rows a call (RHTQ_EINVAL beyond); 65535 sequences and 2^26 - 64 query
 * heads of them all in a query call, 65535 key-value heads (RHTQ_EUNSUPPORTED beyond).
 *
 * The `tokens` new rows belong to sequences by `starts` [seqs+1], ascending from 0: rows starts[s] .. starts[s+1]-1
 * are the last positions of sequence s, up to lengths[s]-1 (lengths count them already).  starts NULL: one row
 * for each sequence (tokens == seqs).  Rows beyond starts[seqs] belong to no sequence; so do positions below 0.
 */
typedef struct {
  uint8_t* k_codes;
  void* k_scales;
  uint8_t* v_codes;
  void* v_scales;
  int32_t layers;     /* page calls: [layers][pages]...; 1 for the others */
  int32_t pages;
  int32_t kv_heads;
  int32_t page;
  int32_t head_dim;
  int32_t scale_dtype;
} rhtq_cache_t;

/* Rotate, quantise and store k, v [tokens][kv_heads][head_dim] (row strides in elements; head_dim contiguous, every row
 * 16-byte aligned).  signs: int8 [head_dim] +-1 or NULL.  Two rows of one call must not fall on the same slot, nor any on a page that
 * sequences share (rhtq_pages_reserve refuses room there).  A row with a value that is not finite gets a NaN scale: it is read as NaN. */
int rhtq_cache_append(const rhtq_cache_t* cache, const void* k, const void* v, int in_dtype, int64_t tokens,
                      int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                      const int32_t* table, int32_t width, const int32_t* lengths, const int32_t* starts, int32_t seqs,
                      const int8_t* k_signs, const int8_t* v_signs, rhtq_stream_t stream);

/* Read rows back: dequantised, rotation undone, to k_out, v_out [tokens][kv_heads][head_dim] contiguous in out_dtype (either may be
 * NULL).  Rows of no sequence or on no page are written as zeros. */
int rhtq_cache_read(const rhtq_cache_t* cache, void* k_out, void* v_out, int out_dtype, int64_t tokens,
                    const int32_t* table, int32_t width, const int32_t* lengths, const int32_t* starts, int32_t seqs,
                    const int8_t* k_signs, const int8_t* v_signs, rhtq_stream_t stream);

/*
 * Attention of one new token per sequence over its cached positions:
 *   o[s][h] = sum_j p_j v_j,  p = softmax_j(scale * q[s][h] . k_j),  j over the visible positions of sequence s,
 * key-value head h / (q_heads / kv_heads).  Visible: every position below lengths[s]; with window > 0 only the last `window`
 * of them and the first `sinks` (window 0: no window, sinks unused).  A sequence with no visible position gets zeros.
 *   q   [seqs][q_heads][head_dim] bf16 or fp16, strides in elements (rows 16-byte aligned); q_heads a multiple of kv_heads
 *   out [seqs][q_heads][head_dim] contiguous, q's type
 *   workspace  rhtq_paged_attention_workspace(...) bytes, 16-byte aligned
 * Scores, softmax and sums are in fp32.  q enters the products as whole numbers, off by at most 2^-22 of a head's largest rotated value,
 * the weights p_j * (scale of v_j) likewise, of the largest among 64 positions.  scale is finite, and scores stay finite in fp32.  A
 * query or a visible value's scale that is not finite, or a visible key's scale that is NaN, gives NaN for the heads that it takes part in.
 * The new token's own row has to be appended first.  8 query heads of a key-value head read the cache once; more read it once for every 8.
 */
int64_t rhtq_paged_attention_workspace(int32_t seqs, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t width,
                                       int32_t page, int32_t window, int32_t sinks);
int rhtq_paged_attention(const void* q, int in_dtype, int32_t seqs, int32_t q_heads, int64_t q_seq_stride,
                         int64_t q_head_stride, const rhtq_cache_t* cache, const int32_t* table, int32_t width,
                         const int32_t* lengths, const int8_t* k_signs, const int8_t* v_signs, float scale, int32_t window,
                         int32_t sinks, void* out, void* workspace, int64_t workspace_bytes, rhtq_stream_t stream);

/*
 * Pages.  refs [pages] int32 counts the table entries that hold a page; 0 = free.  A fresh page is always the lowest free one.
 * The calls that take pages are all or nothing: *status (device int32) is 0 when done, the number of pages missing when there
 * were too few (nothing changed), or -1 when an index, an amount or a length was invalid (nothing changed).
 * workspace: rhtq_pages_workspace(pages, seqs, count) bytes, 16-byte aligned.
 */
int64_t rhtq_pages_workspace(int32_t pages, int32_t seqs, int32_t count);

/* Room for add[s] >= 0 more positions of every sequence: lengths[s] += add[s], fresh pages where table has none (any entry outside
 * [0, pages)), also where the first new position's slot is partly filled and has lost its page: the older positions of such a slot are seen
 * again from then on, and hold nothing until they are appended anew.  Positions beyond width * page count as missing pages.
 * A new position on a page that another entry holds too (refs > 1) is invalid.  It comes about where lengths[s] was lowered below what
 * sequences share: such a sequence is forked at its new length, which gives the fork a page of its own there, and freed. */
int rhtq_pages_reserve(int32_t* table, int32_t width, int32_t* lengths, int32_t seqs, int32_t* refs, int32_t pages,
                       int32_t page, const int32_t* add, int32_t* status, void* workspace, int64_t workspace_bytes,
                       rhtq_stream_t stream);

/* Give up every page of the listed sequences and set their lengths to 0.  Indexes outside [0, seqs) are passed over; one that is
 * listed twice is freed once. */
int rhtq_pages_free(int32_t* table, int32_t width, int32_t* lengths, int32_t seqs, int32_t* refs, int32_t pages,
                    const int32_t* list, int32_t count, rhtq_stream_t stream);

/* Give up the pages that a window (> 0) with its first `sinks` positions can never show again; lengths stay, and count as they do for
 * attention. */
int rhtq_pages_trim(int32_t* table, int32_t width, const int32_t* lengths, int32_t seqs, int32_t* refs, int32_t pages,
                    int32_t page, int32_t window, int32_t sinks, rhtq_stream_t stream);

/* Sequence dst[i] becomes a copy of src[i]: full pages are shared, a partly filled last page is copied (its filled slots, in all
 * layers) to a fresh one.  A src may repeat.  Every dst must be empty (length 0, no pages), listed once and no src. */
int rhtq_pages_fork(const rhtq_cache_t* cache, int32_t* table, int32_t width, int32_t* lengths, int32_t seqs, int32_t* refs,
                    const int32_t* src, const int32_t* dst, int32_t count, int32_t* status, void* workspace,
                    int64_t workspace_bytes, rhtq_stream_t stream);

/* Copy whole pages src[i] -> dst[i] in all layers.  Pairs with an index outside [0, pages) are passed over.  A page that is
 * written twice, or written and read, by one call has undefined bytes. */
int rhtq_pages_copy(const rhtq_cache_t* cache, const int32_t* src, const int32_t* dst, int32_t count, rhtq_stream_t stream);

/* Move live pages (refs > 0) down into the free ones so that they fill [0, live): the i-th live page at or above `live` goes to the i-th free
 * page below it; table and refs follow.  *live (device int32) gets their number. */
int rhtq_pages_compact(const rhtq_cache_t* cache, int32_t* table, int32_t width, int32_t seqs, int32_t* refs, int32_t* live,
                       void* workspace, int64_t workspace_bytes, rhtq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* RHTQ_SERVING_H */
