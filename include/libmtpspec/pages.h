/*
 * libmtpspec, the pages of a draft head's cache between two rounds of drafts: taken, shared, given
 * back and moved together on the device, without a word to the host ([HB] "Rolling back": a KV
 * cache is rolled back by truncation; a row that branches into several drafts goes on from one
 * prefix).  For the caches of latent.h and heads.h alike.  Included by libmtpspec.h, whose
 * conventions hold here.
 *
 * What describes the pages, all int32 on the device:
 *   block_table [B, max_pages]  row b holds the pages block_table[b][0 .. held[b] - 1]
 *   held        [B]             how many
 *   refs        [num_pages]     how many rows hold a page; 0: it is free.  No row holds a page twice.
 * The calls below keep the three in agreement, and set a table's entries that are given back to -1.
 * What each takes and gives depends on no timing: free pages are taken lowest number first, row by
 * row.  1 <= B <= 16384, 1 <= max_pages, num_pages <= 2^31 - 1, 1 <= page_size <= 2^24, and
 * B * max_pages <= 2^40.  Calls on the same description must not overlap.
 */
#ifndef LIBMTPSPEC_PAGES_H
#define LIBMTPSPEC_PAGES_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A further bit of the status word: there were not enough free pages. */
#define MTPSPEC_STATUS_NO_PAGES 0x8

/*
 * mtp_pages_resize — each row keeps what it holds of its first keep[b] positions, and gets room for
 * lens[b] positions that may be written from keep[b] on:
 *   1. every row gives back its pages behind the first ceil(keep[b] / page_size) ones;
 *   2. where the last page kept is partly filled (keep[b] % page_size != 0) and other rows hold it
 *      too, the row leaves it for a page of its own (copy on write): copies[b] = (old, new), to be
 *      given to mtp_pages_copy, and (-1, -1) for all other rows.  If all its holders would leave
 *      it, the lowest row stays;
 *   3. rows take pages up to ceil(lens[b] / page_size).  Pages go to the rows in order, a row's own
 *      last page before its new ones.  From the first row on for which too few are left, rows get
 *      none: they hold what they kept, and MTPSPEC_STATUS_NO_PAGES is OR-ed in.
 * A row with keep[b] < 0 is left as it is.  So is one with a length that does not fit (keep above
 * what is held, lens below keep or above the table); MTPSPEC_STATUS_BAD_PARAM is OR-ed in for it,
 * as for a page id out of range among those of steps 1 and 2, which is passed over.
 *   keep, lens int32 [B]     copies int32 [B, 2], or NULL: step 2 is left out
 *   status     int32 [1] or NULL
 * One launch.
 */
int mtp_pages_resize(const int32_t *keep, const int32_t *lens, int32_t *block_table, int32_t *held,
                     int32_t *refs, int64_t B, int64_t max_pages, int64_t num_pages,
                     int32_t page_size, int32_t *copies, int32_t *status, void *stream);

/*
 * mtp_pages_fork — row dst_rows[i] gives back what it holds and shares the pages of row
 * src_rows[i], for n pairs of rows.  mtp_pages_resize then gives each branch a last page of its own.
 * A row may be the source of many pairs.  A pair is passed over, and MTPSPEC_STATUS_BAD_PARAM OR-ed
 * in, where a row is out of range, where its source is a destination of the call, or where a later
 * pair has the same destination.
 *   src_rows, dst_rows int32 [n], 0 <= n <= 1024     status int32 [1] or NULL
 * One launch.
 */
int mtp_pages_fork(const int32_t *src_rows, const int32_t *dst_rows, int64_t n, int32_t *block_table,
                   int32_t *held, int32_t *refs, int64_t B, int64_t max_pages, int64_t num_pages,
                   int32_t *status, void *stream);

/*
 * mtp_pages_compact — with L pages in use, the ones numbered L and above move into the free numbers
 * below L: the lowest of them into the lowest free one, and so on.  The table and refs are rewritten,
 * and moves lists the pairs (from, to) for mtp_pages_copy, lowest first; afterwards pages 0 .. L - 1
 * are in use and the others free.
 *   moves    int32 [num_pages / 2, 2]; pairs behind the last are set to (-1, -1)
 *   n_moves  int32 [1]: how many there are        status int32 [1] or NULL (a page id out of range)
 * Two launches.
 */
int mtp_pages_compact(int32_t *block_table, const int32_t *held, int32_t *refs, int64_t B,
                      int64_t max_pages, int64_t num_pages, int32_t *moves, int32_t *n_moves,
                      int32_t *status, void *stream);

/*
 * mtp_pages_copy — page to of every cache becomes a copy of page from, for each pair (from, to).
 * The caches of all layers go in one call: page i of caches[c] is the page_bytes bytes at i times
 * page_stride bytes.
 *   caches   host array of n_caches device pointers, 1 <= n_caches <= 64, 16-byte aligned
 *   page_bytes, page_stride  multiples of 16 in bytes, page_bytes <= page_stride
 *   pairs    int32 [n, 2], 0 <= n <= 2^30; a pair with a negative number is passed over; no page is
 *            both copied from and copied to, and none is copied to twice
 *   n_pairs  int32 [1] on the device or NULL: how many of them count (n at most)
 *   status   int32 [1] or NULL: MTPSPEC_STATUS_BAD_PARAM is OR-ed in for a page out of range, whose
 *            pair is passed over
 * One launch.
 */
int mtp_pages_copy(void *const *caches, int32_t n_caches, int64_t num_pages, int64_t page_bytes,
                   int64_t page_stride, const int32_t *pairs, int64_t n, const int32_t *n_pairs,
                   int32_t *status, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBMTPSPEC_PAGES_H */
