/*
 * moe_paged.h - C ABI of the serving path over a paged key/value cache (libmoe.so, GB300 / sm_103a):
 * what runs in front of the routed experts of moe.h in one decode or prompt step.
 *
 *   moe_paged_plan         block tables and slot maps from request lengths
 *   moe_qk_norm_rope       per-head norm and rotation of queries and keys; keys and values to the cache
 *   moe_gqa_paged_decode   attention of one token per sequence (sliding window, sink tokens)
 *   moe_gqa_paged_prefill  attention of many tokens per sequence (prompts, chunks, drafted tokens)
 *   moe_gqa_prefix_decode  attention of one token per sequence behind a prefix all sequences share
 *
 * The cache. k_cache and v_cache are [num_pages, h_kv, page_size, d] bf16, d contiguous, one pair per
 * layer. A sequence's token at position p (counted from 0) is row p % page_size of page
 * block_table[b, p / page_size]; block_table is [B, max_pages] int32 and shared by the layers. A token's
 * slot is page * page_size + p % page_size. page_size is a power of two, 16 .. 1024;
 * num_pages * page_size < 2^31 and num_pages * h_kv < 2^31. The cache itself may be larger than 2^32
 * elements.
 *
 * Which keys a query sees (the masks). A query at position p sees key j when
 *     j <= p   and   (window == 0  or  j > p - window  or  j < n_sink),
 * so window counts the query's own token, window = 0 is full causal attention, and the first n_sink
 * tokens stay visible behind the window. With n_sink >= 0 and window >= 0. A query that sees no key
 * (a sequence of length 0) has out = 0.
 *
 * What may stand in the cache. Rows that no query of the call sees are never used (past a sequence's
 * length, or behind the window of its earliest query): they may hold anything, NaN and infinities
 * included. Pages without a visible row are not read and their block-table entries are not looked at,
 * so pages behind a window can be given to other sequences. Rows that some query of the sequence sees
 * must hold finite values.
 *
 * Numerics: scores and softmax in fp32, 2^x by the hardware's approximation (2^-22 relative),
 * probabilities rounded to bf16 for the probability x value product (the tensor cores take both factors in
 * one type, and values are bf16), sums in fp32, for one token per sequence the last division to 2^-22, the
 * output rounded once to bf16 (nearest even).
 *
 * Conventions: those of moe.h (device pointers owned by the caller, asynchronous on `stream`, host-side
 * checks before any launch, no exceptions across the boundary, graph capturable). Results are
 * deterministic for a given device.
 *
 * Workspace: one zero-filled allocation of moe_paged_workspace_size() bytes (256-byte aligned) serves
 * all calls of one stream, one after the other; every call leaves it ready for the next. Calls that can
 * overlap (other streams, graphs replayed side by side) need workspaces of their own. Its first 4 bytes
 * are a status word that calls set and never clear; zero it to reset it. It keeps the code that matters most: 1-3 before
 * all others, then the largest:
 *   1-3  a kernel gave up a bounded wait (does not happen in correct operation; outputs undefined, zero
 *        the whole workspace before reuse)
 *   4    a length was negative or past the block table (that sequence counts as empty)
 *   6    a visible page's block-table entry was outside [0, num_pages) (its keys and values read as 0)
 *   7    moe_paged_plan left a sequence out: no room in the free list, the table or the token rows
 */
#ifndef MOE_PAGED_H_
#define MOE_PAGED_H_

#include <stddef.h>
#include <stdint.h>

#include "../moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Bytes of workspace the calls of this header need for B sequences with N query tokens in all (N = B for
 * decode) and a shared prefix of prefix_len keys (0 without one). A workspace for larger N, B and prefix_len
 * also serves smaller ones with the same heads. moe_paged_plan needs only the figure for (1, 1, 1, 1, 128, 0). Returns 0 when the
 * sizes are invalid or unsupported. Pure host computation.
 */
size_t moe_paged_workspace_size(int N, int B, int h_q, int h_kv, int d, int prefix_len);

/*
 * Block tables and slot maps of one step, from request lengths.
 *   ctx_lens     [B] int32: tokens each sequence has in the cache, whose ceil(ctx_lens / page_size) pages
 *                stand in its row of block_table
 *   new_lens     [B] int32: tokens it adds in this step (0 is fine)
 *   free_pages   [n_free] int32: the pages nobody owns; the first free_count[0] of them are valid
 *   block_table  [B, max_pages] int32 in/out: rows get their new pages appended; other entries are kept
 *   seq_lens     [B] int32 out: ctx_lens + new_lens, or 0 for a sequence left out
 *   cu_new       [B + 1] int32 out: prefix sum of new_lens (the packed token rows), at most n_rows
 *   positions    [n_rows] int32 out: position of each packed token; 0 behind the last one
 *   slots        [n_rows] int32 out: its slot in the cache; -1 behind the last one and for sequences left out
 *   free_left    [1] int32 out: entries of free_pages still valid; may be free_count itself
 * New pages are taken from the end of the valid part of free_pages, in order of (sequence, page): the k-th
 * is free_pages[free_count - 1 - k]. A sequence is left out (status 7) when the tokens up to and
 * including its own exceed n_rows or its pages the table, or when it needs pages and the pages needed up to and including it (by the sequences
 * in order that fit otherwise) exceed free_count; with a negative length it is left out with status 4 and its
 * new tokens count as 0 when that is the negative one. Sequences left out keep their row of block_table.
 * seq_lens may be ctx_lens itself. A page id outside [0, num_pages) gives slot -1 and status 6.
 * 0 <= B <= 2048 (B = 0 is a no-op), n_rows >= 0, n_free >= 0, max_pages >= 1, B * max_pages < 2^31.
 */
moe_status_t moe_paged_plan(const int32_t* ctx_lens, const int32_t* new_lens, int B, int page_size, int num_pages,
                            const int32_t* free_pages, int n_free, const int32_t* free_count, int32_t* block_table,
                            int max_pages, int32_t* seq_lens, int32_t* cu_new, int32_t* positions, int32_t* slots,
                            int n_rows, int32_t* free_left, void* workspace, size_t ws_bytes, moe_stream_t stream);

/*
 * Norms of queries and keys per head with the position rotation in the same pass; keys and values are stored
 * to the cache.
 *   qkv       [N, (h_q + 2 h_kv) * d] bf16, rows row_stride elements apart (a multiple of 8): per token the
 *             query heads, the key heads, the value heads
 *   q_weight, k_weight  [d] bf16 or null: y = x * rsqrt(mean(x^2) + eps) * weight per head; null: y = x
 *   inv_freq  [rot_dim / 2] f32: pair i of token n turns by the angle positions[n] * inv_freq[i]
 *   rot_dim   leading dimensions that turn, a multiple of 16, 0 .. d. Pair i is dimensions (i, i + rot_dim / 2),
 *             or (2 i, 2 i + 1) when interleaved: (a, b) -> (a cos - b sin, b cos + a sin)
 *   positions [N] int32, slots [N] int32
 *   q_out     [N, h_q, d] bf16 out; must not overlap qkv
 *   k_cache, v_cache  get token n's key and value heads at slots[n]; a token whose slot is outside
 *             [0, num_pages * page_size) is not stored (its q_out is written). Slots of one call are distinct.
 * In fp32 with one rounding to bf16 at the end. The angle is reduced modulo a turn in 64-bit fixed point, so far positions
 * as such lose nothing: it is off by less than |pos| * max(1, |inv_freq|) * 2^-53 turns (the 64-bit rounding of inv_freq in
 * turns). |inv_freq| must be finite. Squares are summed in fp32: a normed row whose squares sum past 2^128 comes out as 0.
 * Values are copied. d = 128, 0 <= N, N = 0 is a no-op.
 */
moe_status_t moe_qk_norm_rope(const uint16_t* qkv, int64_t row_stride, int N, int h_q, int h_kv, int d,
                              const uint16_t* q_weight, const uint16_t* k_weight, float eps, const float* inv_freq,
                              int rot_dim, int interleaved, const int32_t* positions, const int32_t* slots,
                              uint16_t* q_out, uint16_t* k_cache, uint16_t* v_cache, int num_pages, int page_size,
                              moe_stream_t stream);

/*
 * Decode attention over the paged cache: one query token per sequence, at position seq_lens[b] - 1.
 *   q [B, h_q, d] bf16, seq_lens [B] int32 (the new token included), out [B, h_q, d] bf16
 * Heads are grouped as in moe_gqa_decode (query head hq reads key/value head hq / (h_q / h_kv)). Supported:
 * d = 128, h_q a multiple of h_kv, h_q / h_kv <= 16, 0 <= B <= 2048 (B = 0 is a no-op), scale finite. q, the
 * caches and out 16-byte aligned, out apart from all inputs. Work is counted in 32 bits: with N query tokens in
 * all, (N / (2 (128 / G)) + B) * h_kv * (max_pages * page_size / 128 + 9) < 2^31, G = h_q / h_kv. Each visible row
 * is read once per call.
 */
moe_status_t moe_gqa_paged_decode(const uint16_t* q, const uint16_t* k_cache, const uint16_t* v_cache,
                                  const int32_t* block_table, const int32_t* seq_lens, int B, int h_q, int h_kv,
                                  int d, int num_pages, int page_size, int max_pages, float scale, int window,
                                  int n_sink, uint16_t* out, void* workspace, size_t ws_bytes, moe_stream_t stream);

/*
 * Attention of many tokens per sequence over the paged cache (which holds their keys and values already).
 *   q         [N, h_q, d] bf16: packed query tokens; sequence b's are rows cu_q[b] .. cu_q[b + 1] - 1
 *   cu_q      [B + 1] int32, ascending, within 0 .. N
 *   seq_lens  [B] int32: keys of each sequence, its query tokens being the last of them: query i of n sits at
 *             position seq_lens[b] - n + i. Queries at negative positions have out = 0.
 *   out       [N, h_q, d] bf16; rows outside every sequence are left as they were
 * Everything else as in moe_gqa_paged_decode. A cu_q that descends or leaves 0 .. N makes that sequence empty
 * (status 4, its rows are not written). N = 0 or B = 0 is a no-op.
 */
moe_status_t moe_gqa_paged_prefill(const uint16_t* q, const int32_t* cu_q, const uint16_t* k_cache,
                                   const uint16_t* v_cache, const int32_t* block_table, const int32_t* seq_lens, int N,
                                   int B, int h_q, int h_kv, int d, int num_pages, int page_size, int max_pages,
                                   float scale, int window, int n_sink, uint16_t* out, void* workspace,
                                   size_t ws_bytes, moe_stream_t stream);

/*
 * Decode attention behind a prefix that all sequences share: the query of sequence b sees the prefix_len keys
 * in the pages prefix_table [ceil(prefix_len / page_size)] int32 and the seq_lens[b] keys of its own row of
 * block_table (own keys count from 0; seq_lens[b] = 0 is fine). The prefix is computed once for the whole
 * batch, as matrix products over all queries. No window. prefix_len >= 0; with 0 prefix_table may be null.
 * Everything else as in moe_gqa_paged_decode.
 */
moe_status_t moe_gqa_prefix_decode(const uint16_t* q, const int32_t* prefix_table, int prefix_len,
                                   const uint16_t* k_cache, const uint16_t* v_cache, const int32_t* block_table,
                                   const int32_t* seq_lens, int B, int h_q, int h_kv, int d, int num_pages,
                                   int page_size, int max_pages, float scale, uint16_t* out, void* workspace,
                                   size_t ws_bytes, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_PAGED_H_ */
