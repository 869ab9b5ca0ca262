/*
 * moe_kv4.h - C ABI of a paged key/value cache held in 4 bits (libmoe.so, GB300 / sm_103a).
 *
 *   moe_qk_norm_rope_kv4  per-head norm and rotation of queries and keys; keys and values to the cache in 4 bits
 *   moe_gqa_kv4_decode    attention of one token per sequence over it (sliding window, sink tokens)
 *   moe_kv4_load          rows of it back in bf16 pages, for prompts, chunks and drafted tokens
 *                         (moe_gqa_paged_prefill)
 *
 * The cache. One tensor per layer holds keys and values: [num_pages, h_kv, page_size / 16, 2304] bytes, d = 128. Pages,
 * block tables, slots and the masks are those of moe_paged.h. The 2304 bytes of 16 tokens and a head are
 *     keys' codes    16 x 64 bytes
 *     keys' scales   16 x 4 bf16
 *     values' codes  16 x 64 bytes
 *     values' scales 16 x 4 bf16
 * A value is code * scale, with a scale s for 32 consecutive dimensions and codes c in -8 .. 7, held as c + 8. In a
 * token's 64 bytes the 16-bit word 4 g + w holds dimensions 32 w + 4 g .. 32 w + 4 g + 3, the lowest in the lowest 4 bits
 * (g = 0 .. 7, w = 0 .. 3).
 *
 * What is stored for x (already rounded to bf16, as the bf16 cache would hold it): s = max |x| / 7 over the 32
 * dimensions, rounded to bf16, and c = round(x / s) of the exact quotient, halves to even, within -7 .. 7; s = 0 gives
 * c = 0. The error is at most half a scale, a 14th of the group's largest value, and 2^-8 of the value more where the
 * scale was rounded down. A group that holds a NaN or an infinity has a NaN scale and reads back as NaN.
 *
 * Conventions, masks, workspace and status word: those of moe_paged.h (the same workspace serves its calls and these).
 * The cache is 16-byte aligned.
 */
#ifndef MOE_KV4_H_
#define MOE_KV4_H_

#include <stddef.h>
#include <stdint.h>

#include "../moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * moe_qk_norm_rope with the keys and values stored in 4 bits: the codes are of the bf16 values which that call would
 * store. Positions may have several axes, as in moe_qk_norm_mrope (moe_norm.h): with pair_axis null, n_axes is 1 and
 * positions is [N].
 */
moe_status_t moe_qk_norm_rope_kv4(const uint16_t* qkv, int64_t row_stride, int N, int h_q, int h_kv, int d,
                                  const uint16_t* q_weight, const uint16_t* k_weight, float eps,
                                  const float* inv_freq, const int32_t* pair_axis, int rot_dim, int interleaved,
                                  const int32_t* positions, int64_t axis_stride, int n_axes, const int32_t* slots,
                                  uint16_t* q_out, uint8_t* kv4_cache, int num_pages, int page_size,
                                  moe_stream_t stream);

/*
 * moe_gqa_paged_decode over the 4-bit cache: one query token per sequence, at position seq_lens[b] - 1.
 *   q [B, h_q, d] bf16, seq_lens [B] int32 (the new token included), out [B, h_q, d] bf16
 * Numerics: a query's products with the codes are exact, their sums, the scales and the softmax in fp32 (the codes enter as
 * c + 8, the offset is taken off within each group's sum: a score is off by at most 15 * 2^-20 * |scale| * sum |q| s over
 * the dimensions), 2^x to 2^-22 (its argument to 2^-18 where value scales are near the least, 2^-20 for ordinary ones). Each
 * probability times a value scale is rounded once, to fp16 (2^-11 of it), and multiplied with the exact codes into fp32
 * sums; the last division to 2^-22, one rounding to bf16. Products of probability and value scale are held relative to the
 * largest of the sequence: below 2^-20 of it they are off by up to 2^-31 of it instead. Queries are held relative to the
 * largest of their head (2^-100 where that is smaller), exactly down to 2^-20 of it; they may be up to 2^100 in magnitude.
 * Scales are not negative, and those of the values at least 2^-80 or 0. A query that holds a NaN or an infinity gives NaN. A
 * value scale of NaN gives NaN in its dimensions and changes no others, one of the keys' NaN in all of its key/value head's;
 * no scale is infinite (moe_qk_norm_rope_kv4 stores none). Everything else as in moe_gqa_paged_decode.
 */
moe_status_t moe_gqa_kv4_decode(const uint16_t* q, const uint8_t* kv4_cache, const int32_t* block_table,
                                const int32_t* seq_lens, int B, int h_q, int h_kv, int d, int num_pages,
                                int page_size, int max_pages, float scale, int window, int n_sink, uint16_t* out,
                                void* workspace, size_t ws_bytes, moe_stream_t stream);

/*
 * Rows of the 4-bit cache as bf16 rows of another paged cache with the same page size: of sequence b the positions
 * first[b] .. seq_lens[b] - 1 (from 0 with first null), each value code * scale rounded once.
 *   block_table [B, max_pages], dst_table [B, dst_max_pages] int32: the pages of the 4-bit cache and of k_cache and
 *               v_cache [dst_pages, h_kv, page_size, d] bf16. Entries before first[b] / page_size are not looked at.
 * For moe_gqa_paged_prefill over those pages every row that a query sees has to stand there, the context's too, not only the
 * rows that the step adds: first is null, or at most the earliest position that a query of the sequence sees, unless the
 * earlier rows have been read back into these pages before (moe_qk_norm_rope_kv4 does not write them).
 * Other rows of k_cache and v_cache are left as they were. Pages in dst_table are distinct. A length that is negative or
 * past either table, or a negative first, makes that sequence empty (status 4); a source page outside [0, num_pages)
 * reads as zeros, rows for a destination outside [0, dst_pages) are not written (status 6). B as in moe_gqa_paged_decode;
 * B * h_kv * (page_size / 16) * max_pages < 2^31, and the same for dst_max_pages. The workspace need only have
 * moe_paged_workspace_size(1, 1, 1, 1, 128, 0) bytes.
 */
moe_status_t moe_kv4_load(const uint8_t* kv4_cache, const int32_t* block_table, const int32_t* first,
                          const int32_t* seq_lens, int B, int h_kv, int d, int num_pages, int page_size,
                          int max_pages, uint16_t* k_cache, uint16_t* v_cache, const int32_t* dst_table, int dst_pages,
                          int dst_max_pages, void* workspace, size_t ws_bytes, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_KV4_H_ */
