// Attention over the paged latent cache in the absorbed form: every head's query meets the
// cache rows themselves (L latent values and R rotated ones), and the output is the weighted
// sum of the rows' latents.
//
// One pass over the keys with the running maximum m and sum l of a softmax: for a tile of keys
//     S = Q K^T,  p = 2^(s - m),  l += sum p,  O += p V,  and O, l scaled by 2^(m - m') when m
// changes (s, m in powers of two, scale * log2 e folded in).  V is the first L columns of K, so
// a tile is brought to shared memory once and used for both products.  m follows a row's
// maximum only when that has grown by more than 2^8, so O is rarely rescaled.  Weights are rounded
// to 16 bits for the second product; l sums the unrounded ones in fp32.  In fp16, m lies 2^7 below
// the maximum that it was taken from: weights start at 2^7, stay within 2^15, and keep seven more
// powers of two above the subnormal ones; O, l and m carry the factor, and out and lse do not.
//
// Rows: a sequence's T * Hq (token, head) pairs in tiles of 64, which with L <= 512 output
// columns in fp32 take half of the tensor memory (the accumulator of 64 rows is folded into
// 128 lanes x L / 2 columns), so that two score buffers fit beside it.  128 rows would fill it.
// Keys: tiles of 64, 73 KB at L = 512; the ring holds two of them beside the queries.
//
// Work: all units (a row tile against all keys of its sequence) laid end to end in tiles and
// cut evenly over 152 CTAs, one a multiprocessor, whatever the lengths; up to eight CTAs take
// the row tiles of the same keys side by side, so that keys leave HBM once.  A unit cut among
// CTAs leaves fp32 partial outputs, which a second small kernel joins.
//
// What bounds it (bf16, L = 512, R = 64; HBM copy 6.7 TB/s, products 1938 TFLOP/s measured):
//   64 rows a sequence (256 x 500-4000 keys, 725 MB): 148 us, 4.9 TB/s, 0.73 of the copy rate.
//     Counters: DRAM 67 %, tensor pipe 24 %, shared memory of the products 40 %.  The rest is
//     the ends of units, 6,000 cycles each for outputs of 64 rows x 512, and start and join.
//   256 rows a sequence (64 x 1000-8000 keys, 170 GFLOP): 216 us, 0.79 PFLOP/s, 0.41.  A tile
//     takes some 2,750 cycles, 1,792 of them products at the rate of 64-row accumulators,
//     which is set by shared memory (every 16-column step reads 2 KB of queries or weights
//     beside the keys); the keys' arrival and the softmax between the two products take the
//     rest, since a third tile does not fit.
//   168 rows, 100k keys, one sequence: 65 us; as the last, and each row has 50 parts to join.
//   One row of 600 keys: 12 us; 8 x 2k keys, 64 rows: 21 us: two launches and one tile's way
//     from page table to output.
#include <algorithm>

#include "half_types.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace mtpspec {
namespace lat {

using namespace tg;

constexpr int TM = 64;            // (token, head) rows of a unit
constexpr int TN = 64;            // keys of a tile
constexpr int CHUNK = TN * 128;   // bytes of 64 rows x 64 columns of 16 bits
constexpr int MAX_SLOTS = 8;      // the ring of the latents' pieces
constexpr int MAX_ROT_SLOTS = 4;  // and the one of the rotated parts
constexpr int MAX_BOXES = 8;      // boxes of a tile's chunk: pages of at least eight rows
constexpr int RING = 2;           // tiles whose boxes are known: the current and the next
constexpr int NTHREADS = 192;     // warp 0 TMA, warp 1 MMA and TMEM, warps 2-5 softmax
constexpr int SOFTMAX0 = 64;      // the first softmax thread
constexpr int GRID = 152;         // one CTA per SM of a GB300
constexpr float LAZY = 8.0f;      // the running maximum may lag by a factor of 2^8
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr uint32_t POLL_LIMIT = 1u << 25;  // polls of some 20 ns: ~1 s
constexpr int TMEM_COLS = 512;    // output L/2, then scores 2 x 32

struct Params {
    const uint16_t *q;
    int64_t q_row, q_tok, q_head;
    const int32_t *block_table, *kv_len;
    int64_t max_pages;
    int max_len;         // the table's positions, as far as tiles beyond them have 32-bit numbers
    int num_pages, page_size, box_rows;
    int B, T, Hq, L, R;
    int mtiles;          // row tiles of a sequence
    int gs, mgroups;     // CTAs that walk the same keys, one row tile each; such groups a sequence
    int groups;          // groups of CTAs in the grid
    float scale2;  // scale * log2(e), above 0
    uint16_t *out;
    int64_t out_row, out_tok, out_head;
    float *lse;
    int4 *plan;      // what the joining kernel goes by: row, row tile, first and last group of
                     // a unit; by units (wide_join), or by CTAs, the unit that starts in a CTA
                     // and ends in another (row -1 if there is none)
    int wide_join;
    float *part;     // [2 * GRID][rows][L] fp32, normalised partial outputs
    float *part_lse; // [2 * GRID][rows], base 2
    int rows_cap;    // rows of a partial: min(64, T * Hq)
    int32_t *status;
};

__device__ __forceinline__ int row_len(const Params &p, int b) {
    return min(max(p.kv_len[b], 0), p.max_len);
}
__device__ __forceinline__ int tiles_of(int len) { return (len + TN - 1) / TN; }

// An even cut of all units' tiles laid end to end: of the groups that take part, the first
// `rem` have per + 1 tiles, the others per.
struct Cut {
    int64_t total, per;
    int active, rem;
    __device__ __forceinline__ Cut(const Params &p, int64_t tiles) : total(tiles) {
        active = static_cast<int>(tiles < p.groups ? tiles : p.groups);
        if (tiles <= p.groups) {
            per = 1;
            rem = 0;
        } else if (tiles < (int64_t{1} << 31)) {
            per = static_cast<uint32_t>(tiles) / static_cast<uint32_t>(active);
            rem = static_cast<int>(tiles - per * active);
        } else {
            per = tiles / active;
            rem = static_cast<int>(tiles - per * active);
        }
    }
    __device__ __forceinline__ int64_t first(int g) const { return per * g + (g < rem ? g : rem); }
    __device__ __forceinline__ int owner(int64_t tile) const {
        const int64_t big = (per + 1) * rem;
        return static_cast<int>(tile < big ? tile / (per + 1) : rem + (tile - big) / per);
    }
};

// A CTA's walk over its group's tiles, unit by unit; every role walks the same way.
struct Walk {
    int b, mg, off, nt;   // the next unit, the first of its tiles that is ours, its tiles
    int lane;             // which row tile of a unit is this CTA's
    int64_t left;
    int ib, imt, i0, i1, int_, len;  // the current item: row, row tile, tiles i0 .. i1 of int_
    __device__ __forceinline__ bool next(const Params &p) {
        do {
            if (left <= 0) return false;
            while (nt == 0 || off == nt) {  // the next unit
                off = 0;
                if (nt != 0 && ++mg < p.mgroups) break;
                mg = 0;
                if (++b >= p.B) return false;
                len = row_len(p, b);
                nt = tiles_of(len);
            }
            const int n = static_cast<int>(left < nt - off ? left : nt - off);
            ib = b;
            imt = mg * p.gs + lane;
            i0 = off;
            i1 = off + n;
            int_ = nt;
            off += n;
            left -= n;
        } while (imt >= p.mtiles);  // a unit of fewer row tiles than CTAs
        return true;
    }
};

struct __align__(16) Shared {
    uint64_t full[MAX_SLOTS], empty[MAX_SLOTS], rot_full[MAX_ROT_SLOTS], rot_empty[MAX_ROT_SLOTS];
    uint64_t s_full[2], p_ready, pv_done, q_ready, o_empty;
    uint64_t drained;
    float xm[2][4][32];
    int2 box[RING][MAX_BOXES];
    uint32_t tmem;
    volatile int abort;
};

constexpr int SMEM_MAX = 232448;                                        // 227 KB a CTA
constexpr int SMEM_EXTRA = static_cast<int>(sizeof(Shared));

// A bounded wait; once any wait of the CTA has given up, the others return at once, and the
// roles run to their ends without touching what they could not wait for.
__device__ __forceinline__ bool wait(Shared &sh, uint64_t *bar, uint32_t parity,
                                    uint32_t limit = POLL_LIMIT) {
    for (uint32_t it = 0; it < limit; ++it) {
        if (mbar_poll(bar, parity)) return true;
        if (sh.abort) return false;
    }
    sh.abort = 1;
    return false;
}

// The same for a wait that is mostly long: the thread is suspended instead of polling, which
// leaves issue slots and shared memory to the others.
__device__ __forceinline__ bool wait_long(Shared &sh, uint64_t *bar, uint32_t parity,
                                         uint32_t limit = WAIT_LIMIT) {
    for (uint32_t it = 0; it < limit; ++it) {
        if (mbar_test(bar, parity)) return true;
        if (sh.abort) return false;
    }
    sh.abort = 1;
    return false;
}

// Of a CTA that leaves after an abort: the last of a barrier's `fills` lands, or the limit.
__device__ __forceinline__ void wait_out(uint64_t *bar, int fills) {
    for (uint32_t it = 0; fills > 0 && it < WAIT_LIMIT; ++it)
        if (mbar_test(bar, (fills - 1) & 1)) return;
}

// D[64, n] (+)= A[64, 16] B[16, n] with the 64 rows' accumulator folded into 128 lanes: lanes
// 0-63 hold the first n / 2 columns, lanes 64-127 the others.
__device__ __forceinline__ void mma_ws(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.ws.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// The descriptor of a tile whose rows are the products' K axis (the "MN-major" form): its
// 64-column chunks and its groups of 8 rows lie this many bytes apart.
__device__ __forceinline__ uint64_t smem_desc_rows_k(uint32_t addr, uint32_t chunk_step, uint32_t group_step) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(chunk_step >> 4) << 16;
    d |= static_cast<uint64_t>(group_step >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}
template <typename T>
__host__ __device__ constexpr uint32_t idesc_of(int n, bool b_rows_k) {
    return (1u << 4) | (T::mma_format << 7) | (T::mma_format << 10) |
           (static_cast<uint32_t>(b_rows_k) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(TM >> 4) << 24);
}

// What follows from L = 64 NL alone.  The output's columns come in pieces of 256, 128 and 64
// (the widths of the folded accumulator); a slot of the latents' ring holds one piece.
template <int NL>
struct Sizes {
    static constexpr int L = 64 * NL, CHUNKS = NL + 1;  // with the rotated chunk
    static constexpr int PIECES = (NL >> 2) + ((NL >> 1) & 1) + (NL & 1);
    static __host__ __device__ constexpr int first(int k) {  // piece k's first chunk
        return k < (NL >> 2) ? 4 * k : (k == (NL >> 2) && ((NL >> 1) & 1) ? (NL & ~3) : (NL & ~1));
    }
    static __host__ __device__ constexpr int width(int k) {  // its chunks
        return k < (NL >> 2) ? 4 : (k == (NL >> 2) && ((NL >> 1) & 1) ? 2 : 1);
    }
    // Pieces of four chunks lie group by group of 8 rows, the chunks of a group side by side,
    // so that a box of any number of groups is one copy; narrower ones chunk by chunk.
    static __host__ __device__ constexpr int chunk_step(int k) { return width(k) == 4 ? 1024 : CHUNK; }
    static __host__ __device__ constexpr int group_step(int k) { return width(k) == 4 ? 4096 : 1024; }
    static constexpr int COPIES = (NL >> 2) + (NL & 3) + 1;  // of a box of rows, the rotated one too
    static constexpr int UNIT = width(0);
    static constexpr int ROT_SLOTS = NL < 7 ? 4 : 2;
    static constexpr int LEFT = SMEM_MAX - SMEM_EXTRA - (CHUNKS + 1 + ROT_SLOTS) * CHUNK;
    static constexpr int SLOTS = LEFT / (UNIT * CHUNK) < MAX_SLOTS ? LEFT / (UNIT * CHUNK) : MAX_SLOTS;
    static constexpr int SLOT_BYTES = UNIT * CHUNK;
    static constexpr int S_COL = L / 2;  // tensor memory: behind the output
    static constexpr int SMEM = (CHUNKS + 1 + ROT_SLOTS) * CHUNK + SLOTS * SLOT_BYTES + SMEM_EXTRA;
    static_assert(SLOTS > PIECES, "a tile and the start of the next");
};

// The cache's maps.  `wide` sees a page as groups of 8 rows and a row's latents as chunks of 64
// values, and brings four chunks of a box's groups; `one` brings a chunk of a box's rows; `rot`
// the 64 columns from L on, zeros beyond the row's end.
struct Maps {
    CUtensorMap wide, one, rot;
};
template <typename Z>
__device__ __forceinline__ void piece_load(const Maps &m, int k, uint32_t dst, int box, int box_rows,
                                           int row, int page, uint64_t *bar) {
    if (Z::width(k) == 4) {
        tma_load_5d(dst + box * box_rows * 512, &m.wide, 0, 0, Z::first(k), row >> 3, page, bar);
    } else {
#pragma unroll
        for (int c = 0; c < Z::width(k); ++c)
            tma_load_4d(dst + c * CHUNK + box * box_rows * 128, &m.one, 0, row, Z::first(k) + c, page, bar);
    }
}
// The same to L2.
template <typename Z>
__device__ __forceinline__ void piece_prefetch(const Maps &m, int k, int row, int page) {
    if (Z::width(k) == 4) {
        tma_prefetch_5d(&m.wide, 0, 0, Z::first(k), row >> 3, page);
    } else {
#pragma unroll
        for (int c = 0; c < Z::width(k); ++c) tma_prefetch_4d(&m.one, 0, row, Z::first(k) + c, page);
    }
}

template <typename T, int NL>
__global__ void __launch_bounds__(NTHREADS, 1)
k_latent_attn(const __grid_constant__ Maps maps, const Params p) {
    extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle's period
    using Z = Sizes<NL>;
    const uint32_t q_s = smem_addr(smem), p_s = q_s + Z::CHUNKS * CHUNK, kv_s = p_s + CHUNK;
    const uint32_t rot_s = kv_s + Z::SLOTS * Z::SLOT_BYTES;
    Shared &sh = *reinterpret_cast<Shared *>(smem + Z::SMEM - SMEM_EXTRA);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == 0) {
        if (lane < MAX_SLOTS) {
            mbar_init(&sh.full[lane], 1);
            mbar_init(&sh.empty[lane], 1);
        } else if (lane < MAX_SLOTS + MAX_ROT_SLOTS) {
            mbar_init(&sh.rot_full[lane - MAX_SLOTS], 1);
            mbar_init(&sh.rot_empty[lane - MAX_SLOTS], 1);
        } else if (lane == 16) {
            mbar_init(&sh.s_full[0], 1);
            mbar_init(&sh.s_full[1], 1);
            mbar_init(&sh.pv_done, 1);
            mbar_init(&sh.drained, 1);
            sh.abort = 0;
        } else if (lane == 17) {
            mbar_init(&sh.p_ready, 128);
            mbar_init(&sh.q_ready, 128);
            mbar_init(&sh.o_empty, 128);
        } else if (lane == 18) {
            prefetch_map(&maps.wide);
            prefetch_map(&maps.one);
            prefetch_map(&maps.rot);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // (tensor memory is taken only once the kernel before has ended: holding it would stop that
    // kernel's blocks, if they were still to take theirs)
    pdl_wait_primary();
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(&sh.tmem)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // ---- where this CTA starts.  Every warp finds it by itself, from a scan of the rows'
    // tiles with a run of rows a lane: no role waits for another's.
    const int per_lane = (p.B + 31) / 32;
    const int r0 = min(p.B, lane * per_lane), r1 = min(p.B, r0 + per_lane);
    int64_t sum = 0;
    int len_of[8];  // the first eight of them stay in registers
#pragma unroll
    for (int i = 0; i < 8; ++i) len_of[i] = r0 + i < r1 ? row_len(p, r0 + i) : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += tiles_of(len_of[i]);
    for (int b = r0 + 8; b < r1; ++b) sum += tiles_of(row_len(p, b));
    sum *= p.mgroups;
    int64_t at = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, at, o);
        if (lane >= o) at += v;
    }
    const int64_t total = __shfl_sync(0xFFFFFFFFu, at, 31);
    at -= sum;
    const Cut cut(p, total);
    const int cta = blockIdx.x, group = cta / p.gs;
    const int64_t t0 = group < cut.active ? cut.first(group) : total;
    const int64_t t1 = group < cut.active ? cut.first(group + 1) : total;
    Walk w;
    w.left = t1 - t0;
    w.lane = cta - group * p.gs;
    {
        const bool mine = t0 < t1 && at <= t0 && t0 < at + sum;
        int b = r0, n = 0;
        if (mine) {
            bool found = false;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (!found) {
                    n = len_of[i];
                    const int64_t unit_tiles = static_cast<int64_t>(tiles_of(n)) * p.mgroups;
                    found = t0 < at + unit_tiles;
                    if (!found) {
                        at += unit_tiles;
                        ++b;
                    }
                }
            while (!found) {
                n = row_len(p, b);
                const int64_t unit_tiles = static_cast<int64_t>(tiles_of(n)) * p.mgroups;
                found = t0 < at + unit_tiles;
                if (!found) {
                    at += unit_tiles;
                    ++b;
                }
            }
        }
        const int64_t in = t0 - at;  // the row's tiles before it, over all its units
        const unsigned who = __ballot_sync(0xFFFFFFFFu, mine);
        const int src = who ? __ffs(who) - 1 : 0;
        w.b = __shfl_sync(0xFFFFFFFFu, b, src);
        w.len = __shfl_sync(0xFFFFFFFFu, n, src);
        const int64_t off = __shfl_sync(0xFFFFFFFFu, in, src);
        w.nt = tiles_of(w.len);
        w.mg = p.mgroups > 1 && w.nt > 0 ? static_cast<int>(off / w.nt) : 0;
        w.off = static_cast<int>(off - static_cast<int64_t>(w.mg) * w.nt);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;

    if (warp == 0) {
        if (elect_one()) {
            // ---- producer: a tile's pieces, in boxes that stay within a page
            const int boxes = TN / p.box_rows;
            int filled = 0, rot_filled = 0;  // pieces and rotated chunks on their way or there
            int s = 0, rs = 0;               // the next slot of either ring
            uint32_t ph = 1, rph = 1;        // phase of its release
            while (!sh.abort && w.next(p)) {
                const int32_t *table = p.block_table + w.ib * p.max_pages;
                int f = w.i0;  // the next tile to look up: its pages' numbers are being read
                int pi = f * TN / p.page_size, row = f * TN - pi * p.page_size;
                int page[MAX_BOXES], at[MAX_BOXES];
                const auto look = [&]() {
                    int key = f * TN;
#pragma unroll
                    for (int i = 0; i < MAX_BOXES; ++i) {
                        at[i] = row;
                        page[i] = p.num_pages;  // beyond the last page: TMA fills zeros
                        if (i < boxes && key < w.len) {
                            page[i] = table[pi];
                            key += p.box_rows;
                            row += p.box_rows;
                            if (row == p.page_size) {
                                row = 0;
                                ++pi;
                            }
                        }
                    }
                };
                // tile f's boxes are known now (and, with `early`, go to L2)
                const auto settle = [&](bool early) {
                    int first_key = f * TN;
#pragma unroll
                    for (int i = 0; i < MAX_BOXES; ++i) {
                        if (i >= boxes) break;
                        if (first_key < w.len && static_cast<unsigned>(page[i]) >= static_cast<unsigned>(p.num_pages)) {
                            page[i] = p.num_pages;
                            if (p.status) atomicOr(p.status, MTPSPEC_STATUS_BAD_PARAM);
                        }
                        first_key += p.box_rows;
                        sh.box[f % RING][i] = make_int2(page[i], at[i]);
                        if (early) {
#pragma unroll
                            for (int k = 0; k < Z::PIECES; ++k)
                                piece_prefetch<Z>(maps, k, at[i], page[i]);
                            tma_prefetch_3d(&maps.rot, Z::L, at[i], page[i]);
                        }
                    }
                    if (++f < w.i1) look();
                };
                look();
                for (int tile = w.i0; tile < w.i1; ++tile) {
                    if (f <= tile) settle(false);
#pragma unroll
                    for (int k = 0; k < Z::PIECES; ++k) {
                        if (!wait(sh, &sh.empty[s], ph)) break;
                        mbar_expect_tx(&sh.full[s], Z::width(k) * CHUNK);
                        ++filled;
                        const uint32_t dst = kv_s + s * Z::SLOT_BYTES;
#pragma unroll 1
                        for (int i = 0; i < boxes; ++i) {
                            const int2 x = sh.box[tile % RING][i];
                            piece_load<Z>(maps, k, dst, i, p.box_rows, x.y, x.x, &sh.full[s]);
                        }
                        if (++s == Z::SLOTS) {
                            s = 0;
                            ph ^= 1;
                        }
                    }
                    // The next tile goes to L2 as soon as this one's pieces are under way: what
                    // its slots wait for is then the way from L2, which leaves them sooner to
                    // the tile after.  (64 rows x 8k keys x 256 query rows 241 -> 217 us; two
                    // or four tiles ahead 221.)  Pages shorter than a tile multiply the copies:
                    // with 12 a tile it still pays (L = 512, pages of 16, 64 query rows 156 ->
                    // 152 us), with 16 and more it costs (L = 192, pages of 16: 111 -> 115;
                    // L = 512, pages of 8: 156 -> 163).
                    if (boxes * Z::COPIES <= 12 && f < w.i1) settle(true);
                    if (sh.abort || !wait(sh, &sh.rot_empty[rs], rph)) break;
                    mbar_expect_tx(&sh.rot_full[rs], CHUNK);
                    ++rot_filled;
                    uint32_t dst = rot_s + rs * CHUNK;
#pragma unroll 1
                    for (int i = 0; i < boxes; ++i) {
                        const int2 x = sh.box[tile % RING][i];
                        tma_load_3d(dst, &maps.rot, Z::L, x.y, x.x, &sh.rot_full[rs]);
                        dst += p.box_rows * 128;
                    }
                    if (++rs == Z::ROT_SLOTS) {
                        rs = 0;
                        rph ^= 1;
                    }
                }
            }
            pdl_launch_dependents();  // the joining kernel may be set up; it waits for this one
            // after an abort, let the copies in flight land (the last fill of each barrier)
            if (sh.abort) {
                for (int j = 0; j < Z::SLOTS; ++j)
                    wait_out(&sh.full[j], (filled + Z::SLOTS - 1 - j) / Z::SLOTS);
                for (int j = 0; j < Z::ROT_SLOTS; ++j)
                    wait_out(&sh.rot_full[j], (rot_filled + Z::ROT_SLOTS - 1 - j) / Z::ROT_SLOTS);
            }
        }
    } else if (warp == 1) {
        if (elect_one()) {
            // ---- MMA issuer.  Two kinds of work wait for different things: the scores of
            // tile a for its chunks, the products of tile b for its weights.  Whichever is
            // there is issued, the products first, since they free the stage.
            constexpr uint32_t id_qk = idesc_of<T>(TN, false);
            const uint64_t qd = smem_desc_sw128(q_s), pd = smem_desc_sw128(p_s);
            const uint64_t kd = smem_desc_sw128(kv_s), rd = smem_desc_sw128(rot_s);
            int item = 0;
            int sa = 0, sb = 0, ra = 0;            // the next slots of tiles a and b
            uint32_t pa = 0, pra = 0, par = 0;     // their phases; parity of tile a's number
            int ahead = 0;                         // tiles whose scores are issued, products not
            uint32_t pb = 0, idle = 0;             // parity of tile b's number
            bool first = true;                     // tile b is the item's first
            auto products = [&]() {
                if (ahead == 0 || !mbar_poll(&sh.p_ready, pb)) {
                    if (++idle > POLL_LIMIT) sh.abort = 1;
                    return;
                }
                if (first && item > 0 && !wait(sh, &sh.o_empty, (item - 1) & 1)) return;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < Z::PIECES; ++k) {
                    const uint32_t id = idesc_of<T>(Z::width(k) * 64, true);
                    const uint64_t v = smem_desc_rows_k(kv_s, Z::chunk_step(k), Z::group_step(k)) +
                                       sb * (Z::SLOT_BYTES >> 4);
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        mma_ws(tmem + Z::first(k) * 32, pd + 2 * u, v + u * (2 * Z::group_step(k) >> 4), id,
                               !first || u > 0);
                    mma_commit(&sh.empty[sb]);
                    if (++sb == Z::SLOTS) sb = 0;
                }
                mma_commit(&sh.pv_done);
                pb ^= 1;
                --ahead;
                first = false;
                idle = 0;
            };
            // waits for a fill, with products between the polls
            auto filled = [&](uint64_t *bar, uint32_t phase) {
                do {
                    products();
                } while (!mbar_poll(bar, phase) && !sh.abort);
                idle = 0;
                tc_fence_after();
                return !sh.abort;
            };
            while (!sh.abort && w.next(p)) {
                if (!wait(sh, &sh.q_ready, item & 1)) break;
                tc_fence_after();
                first = true;
                for (int tile = w.i0; tile < w.i1 && !sh.abort; ++tile) {
                    while (ahead > 1 && !sh.abort) products();  // the scores' buffer is free
                    const uint32_t d = tmem + Z::S_COL + par * (TN / 2);
                    // chunk c of the queries against the same chunk of the keys
                    const auto scores = [&](int c, uint64_t k) {
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            mma_ws(d, qd + c * (CHUNK >> 4) + 2 * u, k + 2 * u, id_qk, (c | u) != 0);
                    };
#pragma unroll
                    for (int k = 0; k < Z::PIECES; ++k) {
                        if (!filled(&sh.full[sa], pa)) break;
                        // (kd's groups of rows are 1024 bytes apart)
                        const uint64_t key = kd + (static_cast<uint64_t>((Z::group_step(k) - 1024) >> 4) << 32) +
                                             sa * (Z::SLOT_BYTES >> 4);
#pragma unroll
                        for (int i = 0; i < Z::width(k); ++i) scores(Z::first(k) + i, key + i * (Z::chunk_step(k) >> 4));
                        if (++sa == Z::SLOTS) {
                            sa = 0;
                            pa ^= 1;
                        }
                    }
                    if (sh.abort || !filled(&sh.rot_full[ra], pra)) break;
                    scores(NL, rd + ra * (CHUNK >> 4));
                    mma_commit(&sh.s_full[par]);
                    mma_commit(&sh.rot_empty[ra]);
                    if (++ra == Z::ROT_SLOTS) {
                        ra = 0;
                        pra ^= 1;
                    }
                    ++ahead;
                    par ^= 1;
                }
                while (ahead > 0 && !sh.abort) products();
                ++item;
            }
            mma_commit(&sh.drained);
            wait_out(&sh.drained, 1);
        }
    } else {
        // ---- softmax: a pair of threads a row, 32 of a tile's 64 keys each
        const int wq = warp & 3, half = wq >> 1, r = (wq & 1) * 32 + lane;
        const int tid = threadIdx.x - SOFTMAX0;
        const uint32_t trow = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const int vecs = (Z::L + p.R) / 8;
        const int rows_all = p.T * p.Hq;
        int g = 0, slot = 0, piece_slot = 0;
        Walk nw = w;  // one item ahead: its queries are loaded before this item's epilogue
        bool more = nw.next(p);
        auto load_q = [&](const Walk &k) {
            // two threads a row, every other vector each; what lies beyond the row is zero
            const int row = tid >> 1, m = k.imt * TM + row;
            const bool real = m < rows_all;
            const int t = real ? m / p.Hq : 0, h = real ? m - t * p.Hq : 0;
            const uint16_t *src = p.q + (k.ib * p.q_row + t * p.q_tok + h * p.q_head);
            const uint32_t dst = q_s + row * 128;
#pragma unroll 4
            for (int v = tid & 1; v < Z::CHUNKS * 8; v += 2) {
                const bool in = real && v < vecs;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 dst + (v >> 3) * CHUNK + (((v & 7) ^ (row & 7)) << 4)),
                             "l"(in ? src + v * 8 : p.q), "r"(in ? 16 : 0)
                             : "memory");
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_async_smem();
            mbar_arrive(&sh.q_ready);
        };
        if (more) load_q(nw);
        // ---- rows without keys, and lengths out of range, while the first keys are on their way
        for (int b = cta; b < p.B; b += GRID) {
            const int n = p.kv_len[b];
            if (tid == 0 && p.status && (n < 0 || n > p.max_len))
                atomicOr(p.status, MTPSPEC_STATUS_BAD_PARAM);
            if (row_len(p, b) > 0) continue;
            const int row_vecs = Z::L / 8;
            for (int i = tid; i < rows_all * row_vecs; i += 128) {
                const int mm = i / row_vecs, v = i - mm * row_vecs, tt = mm / p.Hq;
                *reinterpret_cast<uint4 *>(p.out + b * p.out_row + tt * p.out_tok +
                                           (mm - tt * p.Hq) * p.out_head + v * 8) =
                    make_uint4(0, 0, 0, 0);
            }
            if (p.lse)
                for (int i = tid; i < rows_all; i += 128)
                    p.lse[static_cast<int64_t>(b) * rows_all + i] = -INFINITY;
        }
        bool cut_here = false;  // a unit starts here and ends in another group
        while (more) {
            w = nw;
            const int m = w.imt * TM + r;
            const int limit = w.len - (p.T - 1 - min(m, rows_all - 1) / p.Hq);
            const int sure = w.len - (p.T - 1 - (w.imt * TM) / p.Hq);  // the least limit
            float m_ref = -INFINITY, l = 0.0f;
            for (int tile = w.i0; tile < w.i1; ++tile, ++g) {
                wait_long(sh, &sh.s_full[g & 1], (g >> 1) & 1);
                tc_fence_after();
                uint32_t x[32];
                tmem_ld32(trow + Z::S_COL + (g & 1) * (TN / 2), x);
                tmem_wait_ld();
                if (__builtin_expect(tile * TN + TN > sure, 0)) {
                    const int seen = limit - (tile * TN + half * 32);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (i >= seen) x[i] = 0xFF800000u;
                }
                float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < 32; i += 2)
                    top4[(i >> 1) & 3] = max3(top4[(i >> 1) & 3], __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
                float top = fmaxf(max3(top4[0], top4[1], top4[2]), top4[3]);
                sh.xm[slot][wq][lane] = top;
                asm volatile("bar.sync %0, 64;" ::"r"(1 + (wq & 1)) : "memory");
                top = fmaxf(top, sh.xm[slot][wq ^ 2][lane]) * p.scale2;
                slot ^= 1;
                const bool raise = top > m_ref + (LAZY + T::first_weight);
                const float m_old = m_ref;
                if (raise) m_ref = top - T::first_weight;
                const float m_use = m_ref == -INFINITY ? 0.0f : m_ref;
                const uint64_t scale_2 = pack2(p.scale2, p.scale2), minus_m = pack2(-m_use, -m_use);
                uint64_t part[2] = {0, 0};  // two pairs of sums
                uint4 weights[4];
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    float e[8];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        float e0, e1;
                        unpack2(fma2(pack2(__uint_as_float(x[8 * v + 2 * u]), __uint_as_float(x[8 * v + 2 * u + 1])),
                                     scale_2, minus_m), e0, e1);
                        e[2 * u] = ex2(e0);
                        e[2 * u + 1] = ex2(e1);
                        part[u & 1] = add2(part[u & 1], pack2(e[2 * u], e[2 * u + 1]));
                    }
                    weights[v] = float_to_half8<T>(e);
                }
                // the products of the tile before are done: the weights' buffer and the
                // output are free to change
                if (g > 0) wait(sh, &sh.pv_done, (g - 1) & 1);
                if (__builtin_expect(tile > w.i0 && __any_sync(0xFFFFFFFFu, raise), 0)) {
                    tc_fence_after();
                    const float f = raise ? ex2(m_old - m_ref) : 1.0f;
                    l *= f;
#pragma unroll 1
                    for (int c = 0; c < Z::L / 2; c += 32) {
                        uint32_t o[32];
                        tmem_ld32(trow + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tmem_st32(trow + c, o);
                    }
                    tmem_wait_st();
                }
                float l0, l1;
                unpack2(add2(part[0], part[1]), l0, l1);
                l += l0 + l1;
                const uint32_t prow = p_s + r * 128;
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                     prow + (((half * 4 + v) ^ (r & 7)) << 4)),
                                 "r"(weights[v].x), "r"(weights[v].y), "r"(weights[v].z),
                                 "r"(weights[v].w)
                                 : "memory");
                if (__builtin_expect(tile * TN + TN > w.len, 0)) {
                    // rows of the tile beyond the sequence: whatever the page holds there
                    // must not meet the zero weights
                    const int z0 = w.len - tile * TN, vec = (TN - z0) * 8;
                    int at = piece_slot;
#pragma unroll
                    for (int k = 0; k < Z::PIECES; ++k) {
                        const uint32_t v = kv_s + at * Z::SLOT_BYTES;
#pragma unroll 1
                        for (int i = tid; i < vec * Z::width(k); i += 128) {
                            const int c = i / vec, in = i - c * vec, z = z0 + (in >> 3);
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                             v + c * Z::chunk_step(k) + (z >> 3) * Z::group_step(k) +
                                             (z & 7) * 128 + (in & 7) * 16),
                                         "r"(0)
                                         : "memory");
                        }
                        if (++at == Z::SLOTS) at = 0;
                    }
                }
                fence_async_smem();
                tc_fence_before();
                mbar_arrive(&sh.p_ready);
                piece_slot += Z::PIECES;
                if (piece_slot >= Z::SLOTS) piece_slot -= Z::SLOTS;
            }
            // ---- this item's scores are all read: its queries may be replaced
            more = nw.next(p);
            if (more) load_q(nw);
            // ---- epilogue
            sh.xm[slot][wq][lane] = l;
            asm volatile("bar.sync %0, 64;" ::"r"(1 + (wq & 1)) : "memory");
            l += sh.xm[slot][wq ^ 2][lane];
            slot ^= 1;
            wait(sh, &sh.pv_done, (g - 1) & 1);
            tc_fence_after();
            const bool whole = w.i0 == 0 && w.i1 == w.int_;
            const bool real = m < rows_all;
            // (a sum of zero: nothing was seen; one that is NaN stays so)
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const float lse2 = l == 0.0f ? -INFINITY : m_ref + log2f(l);
            if (real && half == 0) {
                if (!whole)
                    p.part_lse[(2 * cta + (w.i0 > 0 ? 0 : 1)) * static_cast<int64_t>(p.rows_cap) + r] =
                        lse2;
                else if (p.lse)
                    p.lse[static_cast<int64_t>(w.ib) * rows_all + m] = lse2 * LN2;
            }
            if (tid == 0 && w.i0 == 0 && (!whole || p.wide_join))  // the unit starts here
                p.plan[p.wide_join ? w.ib * p.mtiles + w.imt : cta] = make_int4(
                    w.ib, w.imt, group, cut.owner(t1 - w.left - (w.i1 - w.i0) + w.int_ - 1));
            cut_here |= w.i0 == 0 && !whole;
            // A row a thread: stores of 32 bytes, a whole sector each, where the rows allow it.
            // (The store unit takes a sector of each of 32 rows at a time, 6000 cycles for 64
            // rows; changing places among four lanes first, for whole lines, cost more in
            // shuffles and registers than it saved: 154 -> 175 us in all at 256 rows.)
            const int t = m / p.Hq, h = m - t * p.Hq;
            uint16_t *dst = p.out + w.ib * p.out_row + t * p.out_tok + h * p.out_head;
            float *pdst = p.part + ((2 * cta + (w.i0 > 0 ? 0 : 1)) * static_cast<int64_t>(p.rows_cap) + r) * Z::L;
            const bool sectors = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;
            uint32_t a[2][32];
            tmem_ld32(trow, a[0]);
            int k = 0, c = 0;  // the piece and the accumulator column in its half
#pragma unroll 2
            for (int i = 0; i < NL; ++i) {
                tmem_wait_ld();
                if (i + 1 < NL) tmem_ld32(trow + 32 * (i + 1), a[(i + 1) & 1]);
                const int col = Z::first(k) * 64 + half * (Z::width(k) * 32) + c;
                c += 32;
                if (c == Z::width(k) * 32) {
                    ++k;
                    c = 0;
                }
                if (!real) continue;
                float f[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(a[i & 1][j]) * inv;
                if (whole) {
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        uint32_t x[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = T::narrow2(f[16 * v + 2 * j], f[16 * v + 2 * j + 1]);
                        if (sectors) {
                            st_global_32B(dst + col + 16 * v, x);
                        } else {
                            *reinterpret_cast<uint4 *>(dst + col + 16 * v) = make_uint4(x[0], x[1], x[2], x[3]);
                            *reinterpret_cast<uint4 *>(dst + col + 16 * v + 8) = make_uint4(x[4], x[5], x[6], x[7]);
                        }
                    }
                } else {
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        uint32_t x[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = __float_as_uint(f[8 * v + j]);
                        st_global_32B(pdst + col + 8 * v, x);
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(&sh.o_empty);
        }
        if (!p.wide_join && tid == 0 && !cut_here) p.plan[cta] = make_int4(-1, 0, 0, 0);
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
        if (sh.abort && p.status) atomicOr(p.status, MTPSPEC_STATUS_TIMEOUT);
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(TMEM_COLS)
                     : "memory");
    }
}

// Units cut among groups: each row's partial outputs, weighted by their sums, become the
// output.  With few parts a unit a warp takes a row, and blockIdx.y is the CTA of the first
// kernel in which the unit starts; with many (WIDE), which means few units, a CTA takes a row,
// an eighth of the parts a warp, and blockIdx.y is the unit.
constexpr int JOIN_THREADS = 256, JOIN_WARPS = JOIN_THREADS / 32;

template <typename T, bool WIDE>
__global__ void __launch_bounds__(JOIN_THREADS) k_latent_join(const Params p) {
    __shared__ float sums[WIDE ? JOIN_WARPS : 1][WIDE ? 512 : 1];
    pdl_wait_primary();
    const int4 u = p.plan[blockIdx.y];
    // a row without keys is no unit of the first kernel's
    if (WIDE && row_len(p, blockIdx.y / p.mtiles) == 0) return;
    // (what an aborted call left there is checked)
    if (u.x < 0 || u.x >= p.B || u.y < 0 || u.y >= p.mtiles || u.z < 0 || u.w >= p.groups) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = WIDE ? blockIdx.x : blockIdx.x * JOIN_WARPS + warp;
    const int m = u.y * TM + r, rows_all = p.T * p.Hq, parts = u.w - u.z + 1;
    if (r >= p.rows_cap || m >= rows_all || parts < 2) return;
    // a group's partial of this row: the second slot where the unit starts, else the first
    const int64_t step = static_cast<int64_t>(2) * p.gs * p.rows_cap;
    const int64_t row0 = (static_cast<int64_t>(u.z) * p.gs + u.y % p.gs) * 2 * p.rows_cap + r;
    const auto part_row = [&](int i) { return row0 + i * step + (i == 0 ? p.rows_cap : 0); };
    // every warp finds the row's largest sum by itself
    float top = -INFINITY, sum = 0.0f;
    for (int i = lane; i < parts; i += 32) top = fmaxf(top, p.part_lse[part_row(i)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const float ref = top == -INFINITY ? 0.0f : top;
    // a lane's columns: four of every 128
    float4 acc[4] = {};
    const int first = WIDE ? warp : 0, hop = WIDE ? JOIN_WARPS : 1;
#pragma unroll 2
    for (int i = first; i < parts; i += hop) {
        const int64_t row = part_row(i);
        float4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k * 128 + lane * 4 < p.L)
                v[k] = *reinterpret_cast<const float4 *>(p.part + row * p.L + k * 128 + lane * 4);
        const float w = exp2f(p.part_lse[row] - ref);
        sum += w;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k * 128 + lane * 4 < p.L) {
                acc[k].x += w * v[k].x;
                acc[k].y += w * v[k].y;
                acc[k].z += w * v[k].z;
                acc[k].w += w * v[k].w;
            }
    }
    if (WIDE) {
        __shared__ float warp_sum[JOIN_WARPS];
#pragma unroll
        for (int k = 0; k < 4; ++k) *reinterpret_cast<float4 *>(&sums[warp][k * 128 + lane * 4]) = acc[k];
        if (lane == 0) warp_sum[warp] = sum;
        __syncthreads();
        sum = 0.0f;
#pragma unroll
        for (int w = 0; w < JOIN_WARPS; ++w) sum += warp_sum[w];
        if (warp >= 4) return;
        float4 s4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < JOIN_WARPS; ++w) {
            const float4 x = *reinterpret_cast<const float4 *>(&sums[w][warp * 128 + lane * 4]);
            s4.x += x.x;
            s4.y += x.y;
            s4.z += x.z;
            s4.w += x.w;
        }
        acc[0] = s4;
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int t = m / p.Hq, h = m - t * p.Hq;
    uint16_t *dst = p.out + u.x * p.out_row + t * p.out_tok + h * p.out_head;
#pragma unroll
    for (int k = 0; k < (WIDE ? 1 : 4); ++k) {
        const int col = (WIDE ? warp : k) * 128 + lane * 4;
        if (col < p.L)
            *reinterpret_cast<uint2 *>(dst + col) =
                make_uint2(T::narrow2(acc[k].x * inv, acc[k].y * inv), T::narrow2(acc[k].z * inv, acc[k].w * inv));
    }
    if (p.lse && lane == 0 && (!WIDE || warp == 0))
        p.lse[static_cast<int64_t>(u.x) * rows_all + m] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * LN2;
}

// Diagnostic of the bounded waits, as the other kernels': on a barrier of two arrivals that got
// one, both forms must give up after `limit` polls and raise the abort flag; if not, the timeout
// is taken out of the status word.
__global__ void k_wait_selftest(uint32_t limit, int32_t *status) {
    __shared__ Shared sh;
    if (threadIdx.x != 0) return;
    mbar_init(&sh.drained, 2);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    mbar_arrive(&sh.drained);
    bool ok = true;
    for (int form = 0; form < 2; ++form) {
        sh.abort = 0;
        const bool got = form == 0 ? wait(sh, &sh.drained, 0, limit) : wait_long(sh, &sh.drained, 0, limit);
        ok &= !got && sh.abort;
    }
    if (!ok) atomicAnd(status, ~MTPSPEC_STATUS_TIMEOUT);
}

size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

struct Layout {
    size_t plan, part, lse, total;
    int mtiles, gs, mgroups, rows_cap;
};
Layout layout(int64_t rows, int32_t L) {
    Layout y;
    y.mtiles = static_cast<int>((rows + TM - 1) / TM);
    // CTAs that share their keys walk them side by side, so that the keys leave HBM once;
    // up to eight, in as even groups as there are
    y.mgroups = (y.mtiles + 7) / 8;
    y.gs = (y.mtiles + y.mgroups - 1) / y.mgroups;
    y.rows_cap = static_cast<int>(std::min<int64_t>(rows, TM));
    y.plan = 0;
    y.part = align256(GRID * sizeof(int4));  // (a wide join has fewer units than GRID / 4)
    y.lse = y.part + align256(static_cast<size_t>(2 * GRID) * y.rows_cap * L * 4);
    y.total = y.lse + align256(static_cast<size_t>(2 * GRID) * y.rows_cap * 4);
    return y;
}

template <typename T, int NL>
cudaError_t launch(const Maps &maps, const Params &p, cudaStream_t stream) {
    constexpr int smem = Sizes<NL>::SMEM;
    static AttrCache attr;
    cudaError_t e = ensure_attr(k_latent_attn<T, NL>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem, attr);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(GRID);
    cfg.blockDim = dim3(NTHREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = pdl_attr();  // set up beside the end of whatever the stream runs before
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_latent_attn<T, NL>, maps, p);
    if (e != cudaSuccess) return e;
    count_launches(1);
    cfg.blockDim = dim3(JOIN_THREADS);
    cfg.dynamicSmemBytes = 0;
    cfg.gridDim = p.wide_join ? dim3(p.rows_cap, p.B * p.mtiles)
                              : dim3((p.rows_cap + JOIN_WARPS - 1) / JOIN_WARPS, p.groups * p.gs);
    e = p.wide_join ? cudaLaunchKernelEx(&cfg, k_latent_join<T, true>, p)
             : cudaLaunchKernelEx(&cfg, k_latent_join<T, false>, p);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

template <typename T>
cudaError_t pick(const Maps &maps, const Params &p, cudaStream_t stream) {
    switch (p.L / 64) {
    case 1: return launch<T, 1>(maps, p, stream);
    case 2: return launch<T, 2>(maps, p, stream);
    case 3: return launch<T, 3>(maps, p, stream);
    case 4: return launch<T, 4>(maps, p, stream);
    case 5: return launch<T, 5>(maps, p, stream);
    case 6: return launch<T, 6>(maps, p, stream);
    case 7: return launch<T, 7>(maps, p, stream);
    default: return launch<T, 8>(maps, p, stream);
    }
}

}  // namespace lat

size_t latent_attn_workspace_bytes(int64_t B, int32_t T, int32_t Hq, int32_t L) {
    (void)B;
    return lat::layout(static_cast<int64_t>(T) * Hq, L).total;
}

cudaError_t run_wait_selftest_latent_attn(uint32_t limit, int32_t *status, cudaStream_t stream) {
    lat::k_wait_selftest<<<1, 32, 0, stream>>>(limit, status);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

cudaError_t run_latent_attn(const LatentAttnArgs &a, int dtype, cudaStream_t stream) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    // boxes of the largest power of two (up to a tile) that divides the page: a box never
    // leaves its page, and its rows start at a multiple of eight, the swizzle's period
    const int box = std::min(lat::TN, a.page_size & -a.page_size);
    lat::Maps maps;
    const cuuint64_t W = static_cast<cuuint64_t>(a.L + a.R), P = static_cast<cuuint64_t>(a.page_size);
    const cuuint64_t pages = static_cast<cuuint64_t>(a.num_pages);
    const cuuint64_t page_bytes = static_cast<cuuint64_t>(a.page_stride) * 2;
    const cuuint32_t rows = static_cast<cuuint32_t>(box);
    const auto encode = [&](CUtensorMap *m, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
                            const cuuint32_t *boxes) {
        const cuuint32_t es[5] = {1, 1, 1, 1, 1};
        return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<uint16_t *>(a.cache), dims, strides,
                  boxes, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    const cuuint64_t chunks = static_cast<cuuint64_t>(a.L / 64);
    const cuuint64_t wdims[5] = {64, 8, chunks, P / 8, pages}, wstrides[4] = {W * 2, 128, W * 16, page_bytes};
    const cuuint64_t cdims[4] = {64, P, chunks, pages}, cstrides[3] = {W * 2, 128, page_bytes};
    const cuuint64_t rdims[3] = {W, P, pages}, rstrides[2] = {W * 2, page_bytes};
    const cuuint32_t wide[5] = {64, 8, 4, rows / 8, 1}, one[4] = {64, rows, 1, 1}, rot[3] = {64, rows, 1};
    // (a call encodes the ones that it needs: each costs the host a microsecond)
    const bool quads = a.L >= 256, singles = a.L % 256 != 0;
    if ((quads && !encode(&maps.wide, 5, wdims, wstrides, wide)) ||
        (singles && !encode(&maps.one, 4, cdims, cstrides, one)) || !encode(&maps.rot, 3, rdims, rstrides, rot))
        return cudaErrorInvalidValue;
    if (!quads) maps.wide = maps.one;
    if (!singles) maps.one = maps.wide;
    const lat::Layout y = lat::layout(static_cast<int64_t>(a.T) * a.Hq, a.L);
    unsigned char *ws = static_cast<unsigned char *>(a.workspace);
    lat::Params p = {};
    p.q = a.q;
    p.q_row = a.q_row;
    p.q_tok = a.q_tok;
    p.q_head = a.q_head;
    p.block_table = a.block_table;
    p.kv_len = a.kv_len;
    p.max_pages = a.max_pages;
    p.max_len = static_cast<int>(std::min<int64_t>(a.max_pages * a.page_size, (int64_t{1} << 31) - 256));
    p.num_pages = static_cast<int>(a.num_pages);
    p.page_size = a.page_size;
    p.box_rows = box;
    p.B = static_cast<int>(a.B);
    p.T = a.T;
    p.Hq = a.Hq;
    p.L = a.L;
    p.R = a.R;
    p.mtiles = y.mtiles;
    p.gs = y.gs;
    p.mgroups = y.mgroups;
    p.groups = lat::GRID / y.gs;
    // few units: cut into many parts each, and few rows in all
    p.wide_join = static_cast<int64_t>(p.B) * p.mgroups * 4 < p.groups;
    p.scale2 = a.scale * lat::LOG2E;
    p.out = a.out;
    p.out_row = a.out_row;
    p.out_tok = a.out_tok;
    p.out_head = a.out_head;
    p.lse = a.lse;
    p.plan = reinterpret_cast<int4 *>(ws + y.plan);
    p.part = reinterpret_cast<float *>(ws + y.part);
    p.part_lse = reinterpret_cast<float *>(ws + y.lse);
    p.rows_cap = y.rows_cap;
    p.status = a.status;
    return dtype == MTPSPEC_BF16 ? lat::pick<Bf16>(maps, p, stream) : lat::pick<F16>(maps, p, stream);
}

}  // namespace mtpspec
