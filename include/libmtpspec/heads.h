/*
 * libmtpspec, the draft head's attention with grouped heads: the paged cache of keys and values,
 * and the attention over it ([HB] "The draft head": the block is one full attention layer with
 * norms on its queries and keys, rotary positions and a KV cache of its own, filled by a first
 * pass over the prompt and then a position at a time).  Included by libmtpspec.h, whose
 * conventions hold here; the same block with one shared latent a token is in latent.h.
 *
 * A token has Hq query heads, Hkv key heads and as many value heads of D elements each; query
 * head h goes with key head h / (Hq / Hkv).  Keys and values are kept in pages: position n of
 * row b is at block_table[b][n / page_size], offset n % page_size, of k_cache and of v_cache,
 * which are laid out alike: [num_pages, page_size, Hkv, D] with page, slot and head strides.
 * Elements are 16 bits wide, bfloat16 or float16 (`dtype`), and every array of a call has the
 * same type.  16 <= D <= 256 with D % 16 == 0; Hq a multiple of Hkv, Hq / Hkv <= 128, Hq <= 1024;
 * page_size a multiple of 8, up to 2^24; num_pages and max_pages from 1 to 2^31 - 1.
 *
 * Strides are in elements, multiples of 8, below 2^39, and the last axis is contiguous; 16-bit
 * arrays are 16-byte aligned, whole numbers and floats 4-byte aligned.  An output's axes may
 * come in any order, but no two of its elements may share a place: each stride is at least what
 * the axes of smaller strides span.
 *
 * Cache entries below a row's length, in the pages that its visible positions need, are finite;
 * whatever lies at or beyond the length (an unwritten part of a page, NaN and infinities among it), or
 * in other pages, has no effect.
 */
#ifndef LIBMTPSPEC_HEADS_H
#define LIBMTPSPEC_HEADS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/*
 * mtp_heads_append — T tokens' keys and values into the paged cache, with the heads' norms and
 * rotation in the same pass.  For each token t with row = tok_row[t] and n = positions[t]:
 *     N(x, w) = x / sqrt(mean(x^2) + eps) * w, or x where w is not given   (a head's D elements)
 *     k_cache[block_table[row][n / page_size]][n % page_size][g] = R(n) N(k[t][g], k_norm_w)
 *     v_cache[ ... ][g]                                          = v[t][g]
 *     q_out[t][h] = R(n) N(q[t][h], q_norm_w)                    when q is given
 * R(n) turns the first R elements, as pairs (x_i, y_i), by the angle whose cosine is
 * cos_sin[n][i] and sine cos_sin[n][R/2 + i] (the table holds whatever scaling the positions
 * need); the pairs are elements (2i, 2i + 1) when interleaved is not 0, else (i, R/2 + i).  The
 * other D - R elements stay.  Arithmetic is fp32, each output rounded once.
 *
 *   k, v      [T, Hkv, D] with token and head strides
 *   q, q_out  [T, Hq, D] with token and head strides, or both NULL (Hq is then unused); they may
 *             be the same array
 *   k_norm_w, q_norm_w  [D] or NULL, 16-byte aligned; eps >= 0
 *   cos_sin   float [max_pos, R], 16-byte aligned, contiguous; 16 <= R <= D with R % 16 == 0
 *   tok_row   int32 [T]: the token's row in [0, B); negative: a padding token, skipped
 *   positions int32 [T] in [0, min(max_pos, max_pages * page_size))
 *   block_table int32 [B, max_pages], page ids in [0, num_pages)
 *   status    int32 [1] or NULL: MTPSPEC_STATUS_BAD_PARAM is OR-ed in for a row >= B, a position
 *             out of range or a page id out of range.  Such a token writes nothing to the caches;
 *             its queries are turned all the same when its row and position are good.
 * Tokens of one call have slots of their own.  0 <= T <= 2^20, 1 <= B <= 2^20.  One launch.
 */
int mtp_heads_append(const void *k, int64_t k_tok_stride, int64_t k_head_stride, const void *v,
                     int64_t v_tok_stride, int64_t v_head_stride, const void *k_norm_w,
                     const float *cos_sin, int64_t max_pos, int32_t R, int32_t interleaved,
                     const int32_t *tok_row, const int32_t *positions, int64_t T, int32_t Hkv,
                     int32_t D, const int32_t *block_table, int64_t B, int64_t max_pages,
                     void *k_cache, void *v_cache, int64_t num_pages, int32_t page_size,
                     int64_t page_stride, int64_t slot_stride, int64_t head_stride, const void *q,
                     int64_t q_tok_stride, int64_t q_head_stride, const void *q_norm_w, void *q_out,
                     int64_t q_out_tok_stride, int64_t q_out_head_stride, int32_t Hq, float eps,
                     int dtype, int32_t *status, void *stream);

/*
 * mtp_heads_attn — attention of each row's last tokens over its paged cache: one token a row or
 * 1 + D of them, chunks of prompts, or whole prompts, in any mix.  The queries of all B rows lie
 * one after another: cu_q[b] .. cu_q[b+1] - 1 belong to row b, and are its last positions: with
 * nq of them, query i is at n = kv_len[b] - nq + i (kv_len counts the tokens being processed,
 * whose keys and values are in the cache).  It sees the positions
 *     j <= n,  and with window > 0 of them those with j > n - window or j < sinks
 * (a sliding window, and the first tokens that stay visible).  For each head h:
 *     s_j = scale * q[i][h] . k_cache(b, j)               (D products, fp32)
 *     out[i][h] = sum_j softmax(s)_j v_cache(b, j)
 *     lse[i][h] = ln sum_j e^(s_j)                         (when lse is not NULL)
 * A query that sees nothing (n < 0) has out = 0 and lse = -inf; one with a NaN among the scores
 * that it sees has NaN in both, and changes no other.  The weights are rounded to `dtype` before
 * their products (as the tensor cores take them), all sums are fp32, and the output is rounded
 * once.  In float16 a weight below 2^-21 of the largest one so far has fewer bits than the type's
 * 11, and one below 2^-32 counts for nothing in out (lse has it all the same).
 *
 *   q, out   [Tq, Hq, D] with token and head strides       lse float [Tq, Hq] or NULL
 *   k_cache, v_cache, block_table [B, max_pages] as above; entries of the table that no visible
 *            position needs are not read
 *   cu_q     int32 [B + 1], not decreasing, from 0 to Tq; queries outside every row are not written
 *   kv_len   int32 [B] in [0, min(max_pages * page_size, 2^31 - 256)]
 *   window   0: none, else from 1 on;  sinks >= 0 (without a window it has no effect)
 *   workspace  >= mtp_heads_attn_workspace_bytes(B, Tq, Hq, Hkv, D) bytes, 256-byte aligned; two
 *            calls that may run at the same time need one each
 *   status   int32 [1] or NULL: MTPSPEC_STATUS_BAD_PARAM is OR-ed in for a length out of range
 *            (taken as the nearest in range), a bound out of range or out of order (taken as the
 *            nearest good one: in range, and not below the bounds before it) or a page id out of
 *            range (its positions are read as zeros); MTPSPEC_STATUS_TIMEOUT if a wait gave up.
 * 1 <= B <= 65536, 0 <= Tq <= 2^24, Tq * Hq <= 2^30, scale finite and above 0.  Two launches; the
 * results do not depend on timing.  They may differ in their last bits with the batch that a row is
 * in, since the work is cut among multiprocessors by the lengths of all rows.
 */
int mtp_heads_attn(const void *q, int64_t q_tok_stride, int64_t q_head_stride, const void *k_cache,
                   const void *v_cache, int64_t num_pages, int32_t page_size, int64_t page_stride,
                   int64_t slot_stride, int64_t head_stride, const int32_t *block_table,
                   int64_t max_pages, const int32_t *cu_q, const int32_t *kv_len, int64_t B,
                   int64_t Tq, int32_t Hq, int32_t Hkv, int32_t D, int32_t window, int32_t sinks,
                   float scale, void *out, int64_t out_tok_stride, int64_t out_head_stride,
                   float *lse, int dtype, void *workspace, size_t workspace_bytes, int32_t *status,
                   void *stream);

/* Bytes of device workspace mtp_heads_attn needs; 0 for sizes it would reject, and for Tq == 0.  It
 * depends on D alone: a workspace serves any batch of such heads. */
size_t mtp_heads_attn_workspace_bytes(int64_t B, int64_t Tq, int32_t Hq, int32_t Hkv, int32_t D);

#ifdef __cplusplus
}
#endif

#endif /* LIBMTPSPEC_HEADS_H */
