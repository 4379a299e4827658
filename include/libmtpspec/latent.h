/*
 * libmtpspec, the draft head's latent attention: the paged cache of one latent vector a
 * token, and the attention over it ([ZH] 二.1: the MTP layer's decoder block keeps one shared
 * latent a token; [HB] "The draft head": the block is one attention layer with a KV cache of
 * its own, filled by a first pass over the prompt and then a position at a time).  Included
 * by libmtpspec.h, whose conventions hold here.
 *
 * A token's cache row holds L latent values, which every head shares as key and value, then
 * R values of the key that carry the token's position (rotated by the position's angles).
 * Rows are kept in pages: position n of row b is at block_table[b][n / page_size], offset
 * n % page_size.  Elements are 16 bits wide, bfloat16 or float16 (`dtype`), and every array
 * of a call has the same type.  64 <= L <= 512 with L % 64 == 0; 16 <= R <= 64 with
 * R % 16 == 0; page_size a multiple of 8, up to 2^24; num_pages, max_pages and max_pos from 1
 * to 2^31 - 1.
 *
 * Strides are in elements, multiples of 8, below 2^39, and the last axis is contiguous; 16-bit
 * arrays are 16-byte aligned, whole numbers and floats 4-byte aligned.  An output's axes may
 * come in any order, but no two of its elements may share a place: each stride is at least what
 * the axes of smaller strides span.
 *
 * Cache entries and prompt tokens below a row's length are finite; whatever lies at or
 * beyond it (an unwritten part of a page, NaN and infinities among it) has no effect.
 */
#ifndef LIBMTPSPEC_LATENT_H
#define LIBMTPSPEC_LATENT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The third element type, IEEE half precision: taken by the entry points of this header. */
#define MTPSPEC_F16 2

/*
 * mtp_latent_append — T tokens into the paged cache, their position part rotated on the way.
 * For each token t with row = tok_row[t] and n = positions[t]:
 *     c = latent[t], or rmsnorm(latent[t]) * norm_w when norm_w is given
 *         (rmsnorm(v) = v / sqrt(mean(v^2) + eps))
 *     cache[block_table[row][n / page_size]][n % page_size] = [ c ; R(n) rot[t] ]
 *     q_out[t][h] = R(n) q_rot[t][h]     for every head h, when q_rot is given
 * R(n) turns the pair (x_i, y_i) by the angle whose cosine is cos_sin[n][i] and sine
 * cos_sin[n][R/2 + i]; the pairs are elements (2i, 2i + 1) when interleaved is not 0, else
 * (i, R/2 + i).  Arithmetic is fp32, each output rounded once.
 *
 *   latent    [T, L], row stride latent_stride     rot [T, R], row stride rot_stride
 *   norm_w    [L] or NULL; eps >= 0
 *   cos_sin   float [max_pos, R], 16-byte aligned, contiguous
 *   tok_row   int32 [T]: the token's row in [0, B); negative: a padding token, skipped
 *   positions int32 [T] in [0, min(max_pos, max_pages * page_size))
 *   block_table int32 [B, max_pages], page ids in [0, num_pages)
 *   cache     [num_pages, page_size, L + R], page stride page_stride (rows contiguous)
 *   q_rot, q_out [T, Hq, R] with token and head strides, or both NULL (Hq is then unused);
 *             they may be the same array
 *   status    int32 [1] or NULL: MTPSPEC_STATUS_BAD_PARAM is OR-ed in for a row >= B, a
 *             position out of range or a page id out of range.  Such a token writes nothing
 *             to the cache; its queries are rotated all the same when its row and position
 *             are good.
 * Tokens of one call have slots of their own.  0 <= T <= 2^20, 1 <= B <= 2^20,
 * 1 <= Hq <= 1024.  One launch.
 */
int mtp_latent_append(const void *latent, int64_t latent_stride, const void *rot,
                      int64_t rot_stride, const void *norm_w, float eps, const float *cos_sin,
                      int64_t max_pos, int32_t interleaved, const int32_t *tok_row,
                      const int32_t *positions, int64_t T, int32_t L, int32_t R,
                      const int32_t *block_table, int64_t B, int64_t max_pages, void *cache,
                      int64_t num_pages, int32_t page_size, int64_t page_stride,
                      const void *q_rot, int64_t q_rot_tok_stride, int64_t q_rot_head_stride,
                      void *q_out, int64_t q_out_tok_stride, int64_t q_out_head_stride,
                      int32_t Hq, int dtype, int32_t *status, void *stream);

/*
 * mtp_latent_attn — attention of each row's last T positions over its paged cache, in the
 * absorbed form: the query has been multiplied by the heads' key up-projection, so that it
 * meets the cache rows themselves, and the output is the weighted sum of latents, which the
 * caller multiplies by the value up-projection.  Query t of row b sees the positions
 *     n < kv_len[b] - (T - 1 - t)
 * (kv_len counts the T positions being processed: 1 + D of them in a verification, one in a
 * draft step).  For each head h:
 *     s_n = scale * q[b][t][h] . cache(b, n)          (L + R products, fp32)
 *     out[b][t][h] = sum_n softmax(s)_n cache(b, n)[0..L)
 *     lse[b][t][h] = ln sum_n e^(s_n)                 (when lse is not NULL)
 * A query that sees nothing has out = 0 and lse = -inf; one with a NaN among the scores that it
 * sees has NaN in both, and changes no other.  The weights are rounded to `dtype`
 * before their products (as the tensor cores take them), all sums are fp32, and the output
 * is rounded once.  In float16 a weight below 2^-21 of the largest one so far has fewer bits
 * than the type's 11, and one below 2^-32 counts for nothing in out (lse has it all the same).
 *
 *   q     [B, T, Hq, L + R] with row, token and head strides
 *   out   [B, T, Hq, L] with row, token and head strides      lse float [B, T, Hq] or NULL
 *   cache, block_table, page_size, page_stride, num_pages, max_pages as above; entries of
 *         the table that no visible position needs are not read
 *   kv_len int32 [B] in [0, min(max_pages * page_size, 2^31 - 256)]
 *   workspace  >= mtp_latent_attn_workspace_bytes(B, T, Hq, L, R) bytes, 256-byte aligned
 *   status int32 [1] or NULL: MTPSPEC_STATUS_BAD_PARAM is OR-ed in for a length out of range
 *         (taken as the nearest in range) or a page id out of range (its positions are read
 *         as zeros); MTPSPEC_STATUS_TIMEOUT if a wait gave up.
 * 0 <= B <= 2^20, 1 <= T <= 256, 1 <= Hq <= 1024, T * Hq <= 65536, B * T * Hq <= 2^31 - 1, scale
 * finite and above 0.  Two launches; the results do not depend on timing.
 */
int mtp_latent_attn(const void *q, int64_t q_row_stride, int64_t q_tok_stride,
                    int64_t q_head_stride, const void *cache, int64_t num_pages,
                    int32_t page_size, int64_t page_stride, const int32_t *block_table,
                    int64_t max_pages, const int32_t *kv_len, int64_t B, int32_t T, int32_t Hq,
                    int32_t L, int32_t R, float scale, void *out, int64_t out_row_stride,
                    int64_t out_tok_stride, int64_t out_head_stride, float *lse, int dtype,
                    void *workspace, size_t workspace_bytes, int32_t *status, void *stream);

/* Bytes of device workspace mtp_latent_attn needs; 0 for sizes it would reject. */
size_t mtp_latent_attn_workspace_bytes(int64_t B, int32_t T, int32_t Hq, int32_t L, int32_t R);

/*
 * mtp_latent_prefill — attention over whole prompts in the expanded form: the latents have
 * been multiplied by the up-projections, which gives each head its own N key values and V
 * values a token; the R rotated key values stay shared by the heads.  The tokens of all B
 * sequences lie one after another: queries cu_q[b] .. cu_q[b+1] - 1 and keys cu_k[b] ..
 * cu_k[b+1] - 1 belong to sequence b.  With nq and nk of them, query i sees the keys
 *     j <= i + nk - nq
 * (the sequence's last query sees every key; nk > nq is a chunk behind a cached prefix).
 *     s_j = scale * (q[i][h][0..N) . kv[j][h][0..N) + q[i][h][N..N+R) . rot[j])
 *     out[i][h] = sum_j softmax(s)_j kv[j][h][N..N+V),   lse[i][h] = ln sum_j e^(s_j)
 * A query that sees nothing has out = 0 and lse = -inf; NaN and precision as in mtp_latent_attn.
 *
 *   q    [Tq, Hq, N + R] with token and head strides
 *   kv   [Tk, Hq, N + V] with token and head strides (a token's key, then its value)
 *   rot  [Tk, R], row stride rot_stride, rotated
 *   cu_q, cu_k int32 [B + 1], not decreasing, from 0 to Tq and Tk
 *   out  [Tq, Hq, V] with token and head strides       lse float [Tq, Hq] or NULL
 *   status int32 [1] or NULL: MTPSPEC_STATUS_BAD_PARAM is OR-ed in for a bound out of range
 *        or out of order (taken as the nearest good one: in range, and not below the bounds
 *        before it); MTPSPEC_STATUS_TIMEOUT if a wait gave up.
 * N and V are 64 or 128; 16 <= R <= 64 with R % 16 == 0; 0 <= Tq, Tk <= 2^24 (Tk >= 1 when
 * Tq > 0), 1 <= B <= 65536, 1 <= Hq <= 1024, scale finite and above 0.  Queries outside every
 * sequence are not written.  One launch.
 */
int mtp_latent_prefill(const void *q, int64_t q_tok_stride, int64_t q_head_stride,
                       const void *kv, int64_t kv_tok_stride, int64_t kv_head_stride,
                       const void *rot, int64_t rot_stride, const int32_t *cu_q,
                       const int32_t *cu_k, int64_t B, int64_t Tq, int64_t Tk, int32_t Hq,
                       int32_t N, int32_t R, int32_t V, float scale, void *out,
                       int64_t out_tok_stride, int64_t out_head_stride, float *lse, int dtype,
                       int32_t *status, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBMTPSPEC_LATENT_H */
