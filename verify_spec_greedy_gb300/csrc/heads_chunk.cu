// Attention with grouped heads over the paged cache, for rows of many tokens: chunks of prompts,
// whole prompts, and whatever shares a batch with them.
//
// One pass over the keys with the running maximum m and sum l of a softmax: for a tile of keys
//     S = Q K^T,  p = 2^(s - m),  l += sum p,  O += p V,  and O, l scaled by 2^(m - m') when m
// changes (s, m in powers of two, scale * log2 e folded in; m follows a row's maximum only when
// that has grown by more than 2^8).  Weights are rounded to 16 bits for the second product; l
// sums the unrounded ones in fp32.  (In fp16 m lies 2^7 below that maximum, so that fewer weights
// are subnormal: half_types.cuh.)
//
// Rows: the G = Hq / Hkv query heads of a key head meet the same keys, so a tile's 128 rows are
// TOK = 128 / G tokens times G heads.  A pair of such tiles is a unit of work: while the tensor
// cores work on one tile's products, the other tile's softmax runs, eight warps a tile, two threads
// a row.  Tensor memory holds both tiles' scores (128 columns each, whose first half becomes the
// weights, the left operand of the second product) and outputs.
//
// Keys: tiles of 128 positions, two of them with their values on their way or in use.  A tile is
// brought in boxes that stay within a page, up to sixteen of them, one a lane of the producing
// warp.  With a window, a unit meets the tiles of the first tokens, then those of the window.
//
// Work: all units laid end to end, a unit's length its key tiles and a constant for its start and
// end, and cut evenly over 152 CTAs, one a multiprocessor, whatever the lengths; every CTA finds
// its start from a scan of the rows.  A unit cut among CTAs leaves fp32 partial outputs, which a
// second small kernel joins.
#include <algorithm>

#include "half_types.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace mtpspec {
namespace hch {

using namespace tg;

constexpr int TM = 128;            // (token, head) rows of a tile
constexpr int TN = 128;            // keys of a tile
constexpr int CHUNK = TN * 128;    // bytes of 128 rows x 64 columns of 16 bits
constexpr int NTHREADS = 640;      // warp 0 TMA, 1 MMA, 2 next work, 3 TMEM; 4-11, 12-19 softmax
constexpr int GRID = 152;          // one CTA per SM of a GB300
constexpr int64_t START = 2;       // a unit's start and end, in key tiles
constexpr float LAZY = 8.0f;       // the running maximum may lag by a factor of 2^8
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr uint32_t TMEM_COLS = 512;
constexpr int S_COL = 0, O_COL = 256;  // tile t: + 128 t
constexpr uint32_t POLL_LIMIT = 1u << 25;  // polls of some 20 ns: ~1 s

struct Params {
    const int32_t *cu_q, *kv_len, *block_table;
    int64_t max_pages;
    int max_len;         // the table's positions, up to 2^31 - 256
    int num_pages, page_size, box_rows;
    int B, Tq, Hq, Hkv, G, TOK, D, window, sinks;
    float scale2;        // scale * log2(e), above 0
    uint16_t *out;
    int64_t out_tok, out_head;
    float *lse;
    int4 *plan;          // for the joining kernel, by CTA: the unit that starts there and ends in
                         // another: its first token in q, its tokens, its key head, its parts
    float *part;         // [2 * GRID][2 * TM][64 NC] fp32, normalised partial outputs
    float *part_lse;     // [2 * GRID][2 * TM], base 2
    int32_t *status;
};

__device__ __forceinline__ int row_len(const Params &p, int b) {
    return min(max(p.kv_len[b], 0), p.max_len);
}
// Bound i of cu_q as it is taken: in [0, Tq], and not below the ones before it.
__device__ __forceinline__ int bound(const Params &p, int i, int before) {
    return max(min(p.cu_q[i], p.Tq), before);
}

// A unit: a pair of row tiles of one key head.  first .. : where it starts in its row.
struct Unit {
    int q0, nq, len, tok0;  // the row's first token in q, its tokens and length; the unit's first token
    int w0, ns;             // the first key tile of its window, and the tiles of first tokens before
    __device__ __forceinline__ Unit() {}
    __device__ __forceinline__ Unit(const Params &p, int q0_, int nq_, int len_, int pair)
        : q0(q0_), nq(nq_), len(len_), tok0(pair * 2 * p.TOK) {
        w0 = ns = 0;
        if (p.window > 0 && p.window < len) {
            w0 = max(0, len - nq + tok0 - p.window + 1) / TN;
            ns = min((p.sinks >> 7) + ((p.sinks & 127) != 0), w0);
        }
    }
    // Key tiles that row tile t meets.
    __device__ __forceinline__ int tiles(const Params &p, int t) const {
        const int first = tok0 + t * p.TOK, hi = len - nq + min(first + p.TOK, nq);
        return first >= nq || hi <= 0 ? 0 : ns + ((hi + TN - 1) >> 7) - w0;
    }
    __device__ __forceinline__ int tiles(const Params &p) const { return max(tiles(p, 0), tiles(p, 1)); }
    // Its length in the cut (one tile at least, so that every unit is somebody's).
    __device__ __forceinline__ int64_t weight(const Params &p) const { return START + max(tiles(p), 1); }
};
__device__ __forceinline__ int pairs_of(const Params &p, int nq) { return (nq + 2 * p.TOK - 1) / (2 * p.TOK); }

// An item of a CTA: tiles i0 .. i1 - 1 of a unit's list; with the key tiles before it, and the
// items before it in which either row tile had keys to meet, and the key tiles that it met (as
// far as parities go).  head -1: no more.
struct Item {
    Unit u;
    int row, head, i0, i1, n;   // n: the unit's tiles, at least 1
    uint32_t g0, outputs[2], met[2];
};

struct __align__(16) Shared {
    uint64_t k_full[2], v_full[2], k_free[2], v_free[2];  // by the tile's number mod 2
    uint64_t q_full[2], q_free[2], s_full[2], p_ready[2], o_done[2], v_clean, drained;
    uint64_t item_full[2], item_free[2];
    Item item[2];
    int64_t sums[NTHREADS / 32];
    int64_t total, first_off;
    int first_row, first_q0;
    uint32_t tmem;
    volatile int abort;
    float other[2][2][TM];  // what the two threads of a row tell each other, by tile and half
};

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
// And for one on others whose own waits are bounded, which may take as long as a whole item.
__device__ __forceinline__ bool wait_far(Shared &sh, uint64_t *bar, uint32_t parity,
                                        uint32_t limit = 64 * WAIT_LIMIT) {
    for (uint32_t it = 0; it < limit; ++it) {
        if (mbar_test(bar, parity)) return true;
        if (sh.abort) return false;
    }
    sh.abort = 1;
    return false;
}
// Whether all of two warps that share rows say yes.  They meet at barrier `bar` in everything they
// do, so that after a wait that gave up none may go on without the others.
__device__ __forceinline__ bool both(bool yes, int bar) {
    uint32_t all;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %2, 0;\n\t"
        "bar.red.and.pred p, %1, 64, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(all)
        : "r"(bar), "r"(static_cast<uint32_t>(yes))
        : "memory");
    return all != 0;
}
// The bounded wait of a CTA that leaves, whatever the abort flag says.
__device__ __forceinline__ void wait_out(uint64_t *bar, uint32_t parity) {
    for (uint32_t it = 0; it < WAIT_LIMIT; ++it)
        if (mbar_test(bar, parity)) return;
}

// D[128, n] (+)= A[128, 16] B[16, n], A from tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// A tile whose rows are the products' K axis and whose 64-column chunks are CHUNK apart.
__device__ __forceinline__ uint64_t smem_desc_rows_k(uint32_t addr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(CHUNK >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
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

// An even cut of all units laid end to end: of the CTAs that take part, the first `rem` have
// per + 1, the others per.
struct Cut {
    int64_t total, per;
    int active, rem;
    __device__ __forceinline__ explicit Cut(int64_t sum) : total(sum) {
        active = static_cast<int>(sum < GRID ? sum : GRID);
        per = active > 0 ? sum / active : 0;
        rem = static_cast<int>(sum - per * active);
    }
    __device__ __forceinline__ int64_t first(int g) const {
        return g < active ? per * g + (g < rem ? g : rem) : total;
    }
    __device__ __forceinline__ int owner(int64_t at) const {
        const int64_t big = (per + 1) * rem;
        return static_cast<int>(at < big ? at / (per + 1) : rem + (at - big) / per);
    }
};

// What an item's row tiles and its producer go by.
struct Extent {
    int n0, n1, n, tail;
    __device__ __forceinline__ Extent(const Params &p, const Item &it) {
        n0 = max(0, min(it.i1, it.u.tiles(p, 0)) - it.i0);
        n1 = max(0, min(it.i1, it.u.tiles(p, 1)) - it.i0);
        n = max(n0, n1);
        // the tile that the row's keys end in, if the item meets it and it is not a whole one
        tail = it.u.len % TN != 0 ? it.u.ns + it.u.len / TN - it.u.w0 - it.i0 : -1;
        if (tail >= n) tail = -1;
    }
    __device__ __forceinline__ int tiles(int t) const { return t ? n1 : n0; }
    // the tile of rows that uses every chunk last
    __device__ __forceinline__ int last() const { return n1 >= n0 ? 1 : 0; }
};
// The number of the unit's i-th key tile.
__device__ __forceinline__ int key_tile(const Unit &u, int i) { return i < u.ns ? i : i - u.ns + u.w0; }

template <int NC>
struct Sizes {
    static constexpr int TILE = 2 * NC, RING = 2 * TILE;   // chunks of a tile's keys and values
    static constexpr int EXTRA = static_cast<int>(sizeof(Shared));
    // (more than half of an SM's, so that no two CTAs, which take all its tensor memory, share one)
    static constexpr int SMEM = ((2 * NC + RING) * CHUNK > 120 * 1024 ? (2 * NC + RING) * CHUNK : 120 * 1024) + EXTRA;
    static constexpr int COLS = 64 * NC;
};

struct Maps {
    CUtensorMap q, k, v;
};

// NC: the 64-column chunks of a head.
template <typename T, int NC>
__global__ void __launch_bounds__(NTHREADS, 1)
k_heads_chunk(const __grid_constant__ Maps maps, const Params p) {
    extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle's period
    using Z = Sizes<NC>;
    const uint32_t q_s = smem_addr(smem), ring = q_s + 2 * NC * CHUNK;
    Shared &sh = *reinterpret_cast<Shared *>(smem + Z::SMEM - Z::EXTRA);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(&sh.q_full[t], 1);
            mbar_init(&sh.q_free[t], 1);
            mbar_init(&sh.k_full[t], 1);
            mbar_init(&sh.v_full[t], 1);
            mbar_init(&sh.k_free[t], 1);
            mbar_init(&sh.v_free[t], 1);
            mbar_init(&sh.s_full[t], 1);
            mbar_init(&sh.p_ready[t], 256);
            mbar_init(&sh.o_done[t], 1);
            mbar_init(&sh.item_full[t], 1);
            mbar_init(&sh.item_free[t], 18);  // the producer, the issuer, sixteen softmax warps
        }
        mbar_init(&sh.v_clean, 256);
        mbar_init(&sh.drained, 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&maps.q);
        prefetch_map(&maps.k);
        prefetch_map(&maps.v);
    }
    // (tensor memory is taken only once the kernel before has ended: holding it would stop that
    // kernel's blocks, if they were still to take theirs)
    pdl_wait_primary();
    if (warp == 3) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(&sh.tmem)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // ---- where this CTA starts: a scan of the rows' units, a run of rows a thread, or, of few
    // rows, a row a warp whose lanes share its units
    const bool wide = p.B <= NTHREADS / 32;
    const int run = wide ? 1 : (p.B + NTHREADS - 1) / NTHREADS;
    const int b0 = min(p.B, wide ? warp : static_cast<int>(threadIdx.x) * run), b1 = min(p.B, b0 + run);
    bool bad = false, order = false;
    for (int b = b0; b < b1; ++b) {
        const int c0 = p.cu_q[b], c1 = p.cu_q[b + 1], len = p.kv_len[b];
        order |= c0 < 0 || c1 > p.Tq || c1 < c0;
        bad |= len < 0 || len > p.max_len;
    }
    const bool disorder = __syncthreads_or(order);
    if (__syncthreads_or(bad || order) && blockIdx.x == 0 && threadIdx.x == 0 && p.status)
        atomicOr(p.status, MTPSPEC_STATUS_BAD_PARAM);
    int q_before = 0;  // the largest bound up to the first of the run, as taken
    if (disorder)
        for (int b = 0; b < b0; ++b) q_before = bound(p, b, q_before);
    int64_t sum = 0;
    {
        int q0 = b0 < b1 ? bound(p, b0, q_before) : 0;
        for (int b = b0; b < b1; ++b) {
            const int q1 = bound(p, b + 1, q0), len = row_len(p, b);
            const int pairs = pairs_of(p, q1 - q0);
            for (int i = wide ? lane : 0; i < pairs; i += wide ? 32 : 1)
                sum += Unit(p, q0, q1 - q0, len, i).weight(p);
            q0 = q1;
        }
    }
    sum *= p.Hkv;
    int64_t at = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, at, o);
        if (lane >= o) at += v;
    }
    if (lane == 31) sh.sums[warp] = at;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < NTHREADS / 32; ++w) {
        if (w == warp) at += total;
        total += sh.sums[w];
    }
    at -= sum;
    const Cut cut(total);
    const int64_t t0 = cut.first(blockIdx.x), t1 = cut.first(blockIdx.x + 1);
    if (wide) {  // the row's sum is its whole warp's
        at = __shfl_sync(0xFFFFFFFFu, at, 0);
        sum = sh.sums[warp];
    }
    if (t0 < t1 && at <= t0 && t0 < at + sum && (!wide || lane == 0)) {
        int q0 = bound(p, b0, q_before), b = b0;
        int64_t off = t0 - at;
        for (; b + 1 < b1; ++b) {  // (a run of one row has nothing to look for)
            const int q1 = bound(p, b + 1, q0), len = row_len(p, b);
            int64_t mine = 0;
            for (int i = 0; i < pairs_of(p, q1 - q0); ++i) mine += Unit(p, q0, q1 - q0, len, i).weight(p);
            mine *= p.Hkv;
            if (off < mine) break;
            off -= mine;
            q0 = q1;
        }
        sh.first_row = b;
        sh.first_q0 = q0;
        sh.first_off = off;
    }
    __syncthreads();
    // ---- the scheduler's walk (warp 2, all lanes alike): the unit `pair` of key head `head` of row
    // `row`, which starts at `a` in the cut, and what is left from `cur` on
    int row = 0, q0 = 0, q1 = 0, len = 0, head = 0, pair = 0, pairs = 0;
    int64_t cur = t0, a = t0;
    bool cut_here = false;
    const auto open_row = [&]() {
        q1 = bound(p, row + 1, q0);
        len = row_len(p, row);
        pairs = pairs_of(p, q1 - q0);
    };
    // the next item that has tiles; false if there is none
    const auto next = [&](Item &it) {
        while (cur < t1) {
            while (pair >= pairs) {  // (rows without tokens have no units)
                pair = 0;
                if (pairs == 0 || ++head == p.Hkv) {
                    head = 0;
                    q0 = q1;
                    if (++row >= p.B) return false;
                    open_row();
                }
            }
            it.u = Unit(p, q0, q1 - q0, len, pair);
            it.n = max(it.u.tiles(p), 1);
            it.row = row;
            it.head = head;
            const int64_t base = a + START, s = max(cur, base), e = min(t1, base + it.n);
            a = base + it.n;
            cur = min(t1, a);
            ++pair;
            if (s >= e) continue;
            it.i0 = static_cast<int>(s - base);
            it.i1 = static_cast<int>(e - base);
            if (it.i0 == 0 && it.i1 < it.n && lane == 0) {
                cut_here = true;
                p.plan[blockIdx.x] = make_int4(q0 + it.u.tok0, min(2 * p.TOK, q1 - q0 - it.u.tok0), head,
                                               cut.owner(base + it.n - 1) - static_cast<int>(blockIdx.x) + 1);
            }
            return true;
        }
        return false;
    };
    if (warp == 2) {
        Item it = {};
        it.head = -1;
        if (t0 < t1) {
            row = sh.first_row;
            q0 = sh.first_q0;
            open_row();
            // the row's units of one head, 32 at a time, until the one that t0 lies in
            int64_t off = sh.first_off, mine = 0;
            for (int i = lane; i < pairs; i += 32) mine += Unit(p, q0, q1 - q0, len, i).weight(p);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, o);
            head = static_cast<int>(off / mine);
            off -= head * mine;
            for (pair = 0;; pair += 32) {
                const int i = pair + lane;
                const int64_t w = i < pairs ? Unit(p, q0, q1 - q0, len, i).weight(p) : 0;
                int64_t to = w;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t v = __shfl_up_sync(0xFFFFFFFFu, to, o);
                    if (lane >= o) to += v;
                }
                const int64_t here = __shfl_sync(0xFFFFFFFFu, to, 31);
                if (off < here || pair + 32 >= pairs) {
                    const unsigned who = __ballot_sync(0xFFFFFFFFu, off < to);
                    const int src = who ? __ffs(who) - 1 : 0;
                    off -= __shfl_sync(0xFFFFFFFFu, to - w, src);
                    pair += src;
                    break;
                }
                off -= here;
            }
            a = t0 - off;
            if (!next(it)) it.head = -1;
        }
        if (lane == 0) sh.item[0] = it;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    // Every role goes through the CTA's items: is there one after number `item`, and no abort?
    const auto next_item = [&](uint32_t item) {
        ++item;
        return wait_far(sh, &sh.item_full[item & 1], ((item - 1) >> 1) & 1) && sh.item[item & 1].head >= 0;
    };

    if (sh.item[0].head < 0) {
        // nothing: fewer tiles than CTAs
    } else if (warp >= 4) {
        // ---- softmax: two threads a row, 64 of a tile's 128 keys each
        const int t = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1, r = (warp & 3) * 32 + lane;
        const uint32_t lane_bits = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_t = tmem + lane_bits + S_COL + t * 128, o_t = tmem + lane_bits + O_COL + t * 128;
        const int pair_bar = 1 + t * 4 + (warp & 3);
        const int my_tok = r / p.G;  // within the tile
        // this thread's value for the row's other thread, and the other's
        const auto swap = [&](float v) {
            sh.other[t][half][r] = v;
            asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory");
            return sh.other[t][half ^ 1][r];
        };
        for (uint32_t item = 0;; ++item) {
            // (what only the item's end needs stays in shared memory meanwhile)
            const volatile Item &my = sh.item[item & 1];
            int nt, tail, limit, sure, width;  // limit: one past the last key that this row sees
            int ns, skip, i0;
            {
                Item it;
                it.u.nq = my.u.nq;
                it.u.len = my.u.len;
                it.u.tok0 = my.u.tok0;
                it.u.w0 = my.u.w0;
                it.u.ns = my.u.ns;
                it.i0 = i0 = my.i0;
                it.i1 = my.i1;
                const Extent e(p, it);
                nt = e.tiles(t);
                tail = e.last() == t ? e.tail : -1;  // the tile whose values are to be cleared
                sure = it.u.len - it.u.nq + it.u.tok0 + t * p.TOK + 1;  // the least limit of the tile's rows
                limit = sure + my_tok;
                width = p.window > 0 && p.window < it.u.len ? p.window : 0;
                ns = it.u.ns;
                skip = it.u.w0 - ns;
            }
            uint32_t parity = my.met[t] & 1;
            float m_ref = -INFINITY, l = 0.0f;
            for (int j = 0; j < nt; ++j) {
                wait_long(sh, &sh.s_full[t], parity);
                parity ^= 1;
                tc_fence_after();
                uint32_t x[2][32];
                tmem_ld32(s_t + half * 64, x[0]);
                tmem_ld32(s_t + half * 64 + 32, x[1]);
                if (__builtin_expect(j == tail, 0)) {
                    // value rows behind the row's last key: whatever lies there must not meet the
                    // zero weights.  (The barrier's fill before this one is used up by now, so
                    // the phase is this fill's.)
                    const uint32_t g = my.g0 + tail;
                    wait(sh, &sh.v_full[g & 1], (g >> 1) & 1);
                    const int z0 = my.u.len % TN;
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        const uint32_t v = ring + ((g & 1) * Z::TILE + NC + c) * CHUNK + z0 * 128;
                        for (int i = half * 128 + r; i < (TN - z0) * 8; i += 256)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(v + i * 16), "r"(0)
                                         : "memory");
                    }
                    fence_async_smem();
                    mbar_arrive(&sh.v_clean);
                }
                tmem_wait_ld();
                const int key0 = (i0 + j < ns ? i0 + j : i0 + j + skip) * TN;
                if (__builtin_expect(key0 + TN > sure || (width && key0 < sure + p.TOK - 1 - width), 0)) {
                    // more than every row sees
                    const int seen = limit - key0 - half * 64;
                    const int low = width ? seen - width : -1, first = p.sinks - key0 - half * 64;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        if (i >= seen || (i < low && i >= first)) x[0][i] = 0xFF800000u;
                        if (i + 32 >= seen || (i + 32 < low && i + 32 >= first)) x[1][i] = 0xFF800000u;
                    }
                }
                float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    top4[i & 3] = max3(top4[i & 3], __uint_as_float(x[0][i]), __uint_as_float(x[1][i]));
                const float mine = fmaxf(max3(top4[0], top4[1], top4[2]), top4[3]);
                // (the second barrier of a tile is p_ready: nobody writes the next value before
                // the products have taken both threads' weights)
                const float top = fmaxf(mine, swap(mine)) * p.scale2;
                const bool raise = top > m_ref + (LAZY + T::first_weight);
                const float m_new = top - T::first_weight;
                if (__builtin_expect(j > 0 && __any_sync(0xFFFFFFFFu, raise), 0)) {
                    // the scores came after the products of the tile before: the output is free
                    const float f = raise ? ex2(m_ref - m_new) : 1.0f;
                    l *= f;
#pragma unroll
                    for (int c = half * (NC * 32); c < (half + 1) * (NC * 32); c += 16) {
                        uint32_t o[16];
                        tmem_ld16(o_t + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tmem_st16(o_t + c, o);
                    }
                }
                if (raise) m_ref = m_new;
                const float m_use = m_ref == -INFINITY ? 0.0f : m_ref;
                const uint64_t scale_2 = pack2(p.scale2, p.scale2), minus_m = pack2(-m_use, -m_use);
                uint64_t part[2] = {0, 0};  // two pairs of sums
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float e0, e1;
                        unpack2(fma2(pack2(__uint_as_float(x[c][2 * i]), __uint_as_float(x[c][2 * i + 1])),
                                     scale_2, minus_m), e0, e1);
                        e0 = ex2(e0);
                        e1 = ex2(e1);
                        part[i & 1] = add2(part[i & 1], pack2(e0, e1));
                        w[i] = T::narrow2(e0, e1);
                    }
                    tmem_st16(s_t + half * 32 + 16 * c, w);
                }
                tmem_wait_st();
                float l0, l1;
                unpack2(add2(part[0], part[1]), l0, l1);
                l += l0 + l1;
                tc_fence_before();
                mbar_arrive(&sh.p_ready[t]);
            }
            if (nt > 0) {
                wait_long(sh, &sh.o_done[t], my.outputs[t] & 1);
                tc_fence_after();
            }
            l += swap(l);
            // (a sum of zero: nothing was seen; one that is NaN stays so)
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const float lse2 = l == 0.0f ? -INFINITY : m_ref + log2f(l);
            const int tok = my.u.tok0 + t * p.TOK + my_tok, h = my.head * p.G + r - my_tok * p.G;
            const bool real = my_tok < p.TOK && tok < my.u.nq;
            const bool whole = my.i0 == 0 && my.i1 == my.n;
            const int64_t out_row = my.u.q0 + tok;
            const int64_t part_row = static_cast<int64_t>(2 * blockIdx.x + (my.i0 > 0 ? 0 : 1)) * (2 * TM) +
                                     t * TM + r;
            if (real && half == 0) {
                if (!whole)
                    p.part_lse[part_row] = lse2;
                else if (p.lse)
                    p.lse[out_row * p.Hq + h] = lse2 * LN2;
            }
            uint16_t *dst = p.out + out_row * p.out_tok + h * p.out_head + half * (NC * 32);
            float *pdst = p.part + part_row * Z::COLS + half * (NC * 32);
            // 32 bytes a store, a whole sector, where the rows allow it
            const bool sectors = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                uint32_t o[32] = {};
                if (nt > 0) {
                    tmem_ld32(o_t + half * (NC * 32) + 32 * c, o);
                    tmem_wait_ld();
                }
                if (!real) continue;
                if (!whole) {
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        uint32_t y[8];
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            y[u] = nt > 0 ? __float_as_uint(__uint_as_float(o[8 * v + u]) * inv) : 0u;
                        st_global_32B(pdst + c * 32 + v * 8, y);
                    }
                    continue;
                }
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    if (half * (NC * 32) + c * 32 + v * 16 >= p.D) break;
                    uint32_t y[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        y[u] = nt > 0 ? T::narrow2(__uint_as_float(o[16 * v + 2 * u]) * inv,
                                                   __uint_as_float(o[16 * v + 2 * u + 1]) * inv)
                                      : 0u;
                    uint16_t *d = dst + c * 32 + v * 16;
                    if (sectors) {
                        st_global_32B(d, y);
                    } else {
                        *reinterpret_cast<uint4 *>(d) = make_uint4(y[0], y[1], y[2], y[3]);
                        *reinterpret_cast<uint4 *>(d + 8) = make_uint4(y[4], y[5], y[6], y[7]);
                    }
                }
            }
            // The next item's products overwrite this output once its first weights are there,
            // which come after these reads.
            tc_fence_before();
            __syncwarp();  // the whole warp is done with the item
            if (lane == 0) mbar_arrive(&sh.item_free[item & 1]);
            if (!both(next_item(item), pair_bar)) break;
        }
    } else if (warp == 0) {
        // ---- producer: a box of a tile a lane.  Tiles are numbered through all items of the CTA,
        // and tile j takes the half j mod 2 of the ring.
        const int boxes = TN / p.box_rows;
        const uint32_t q_bytes = NC * p.G * p.TOK * 128;
        uint32_t j = 0, q_uses[2] = {0, 0};
        const auto all = [](bool yes) { return __all_sync(0xFFFFFFFFu, yes) != 0; };
        for (uint32_t item = 0;; ++item) {
            const Item my = sh.item[item & 1];
            const Extent x(p, my);
            // the page of this lane's box of the item's tile i
            const int32_t *table = p.block_table + static_cast<int64_t>(my.row) * p.max_pages;
            int page = 0, slot = 0;
            const auto look = [&](int i) {
                const int key = key_tile(my.u, my.i0 + i) * TN + lane * p.box_rows;
                const int pi = key / p.page_size;
                slot = key - pi * p.page_size;
                page = p.num_pages;  // beyond the last page: TMA fills zeros
                if (lane < boxes && key < my.u.len) {
                    page = table[pi];
                    if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_pages)) {
                        page = p.num_pages;
                        if (p.status) atomicOr(p.status, MTPSPEC_STATUS_BAD_PARAM);
                    }
                }
            };
            if (x.n > 0) look(0);
            bool ok = true;
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if (ok && x.tiles(t) > 0) {
                    if (q_uses[t] > 0 && !all(wait(sh, &sh.q_free[t], (q_uses[t] - 1) & 1))) {
                        ok = false;
                        break;
                    }
                    ++q_uses[t];
                    if (lane == 0) {
                        mbar_expect_tx(&sh.q_full[t], q_bytes);
                        for (int c = 0; c < NC; ++c)
                            tma_load_4d(q_s + (t * NC + c) * CHUNK, &maps.q, c * 64, 0,
                                        my.u.q0 + my.u.tok0 + t * p.TOK, my.head, &sh.q_full[t]);
                    }
                    __syncwarp();
                }
            for (int i = 0; ok && i < x.n; ++i, ++j) {
                const int to_page = page, to_slot = slot;
                if (i + 1 < x.n) look(i + 1);
                const uint32_t half = j & 1, before = ((j >> 1) - 1) & 1;
                const uint32_t dst = ring + half * (Z::TILE * CHUNK) + lane * p.box_rows * 128;
                if (j > 1 && !all(wait(sh, &sh.k_free[half], before))) {
                    ok = false;
                    break;
                }
                if (lane == 0) mbar_expect_tx(&sh.k_full[half], NC * CHUNK);
                __syncwarp();
                if (lane < boxes)
                    for (int c = 0; c < NC; ++c)
                        tma_load_4d(dst + c * CHUNK, &maps.k, c * 64, my.head, to_slot, to_page, &sh.k_full[half]);
                __syncwarp();
                if (j > 1 && !all(wait(sh, &sh.v_free[half], before))) {
                    ++j;  // (its keys are on their way)
                    ok = false;
                    break;
                }
                if (lane == 0) mbar_expect_tx(&sh.v_full[half], NC * CHUNK);
                __syncwarp();
                if (lane < boxes)
                    for (int c = 0; c < NC; ++c)
                        tma_load_4d(dst + (NC + c) * CHUNK, &maps.v, c * 64, my.head, to_slot, to_page,
                                    &sh.v_full[half]);
                __syncwarp();
            }
            if (!ok || !all(!sh.abort)) break;
            if (lane == 0) mbar_arrive(&sh.item_free[item & 1]);
            if (!all(next_item(item))) break;
        }
        if (__any_sync(0xFFFFFFFFu, sh.abort)) {
            // let the copies in flight land: the last two tiles' and the queries' (a fill that was
            // cut off never completes: its wait runs to the limit)
            for (uint32_t i = j > 2 ? j - 2 : 0; i < j; ++i) {
                wait_out(&sh.k_full[i & 1], (i >> 1) & 1);
                wait_out(&sh.v_full[i & 1], (i >> 1) & 1);
            }
            for (int t = 0; t < 2; ++t)
                if (q_uses[t] > 0) wait_out(&sh.q_full[t], (q_uses[t] - 1) & 1);
        }
    } else if (warp == 1) {
        if (elect_one()) {
            // ---- MMA issuer: a tile's products, then its next scores, in turn
            constexpr uint32_t id_s = idesc_of<T>(TN, false);
            constexpr uint32_t id_o = idesc_of<T>(NC * 64, true);
            const uint64_t qd = smem_desc_sw128(q_s), kd = smem_desc_sw128(ring);
            const uint64_t vd = smem_desc_rows_k(ring) + NC * (CHUNK >> 4);
            const auto scores = [&](uint32_t g, int t) {
                const uint32_t d = tmem + S_COL + t * 128;
                const uint64_t a_d = qd + t * (NC * (CHUNK >> 4));
                const uint64_t b_d = kd + (g & 1) * (Z::TILE * (CHUNK >> 4));
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        mma_bf16(d, a_d + c * (CHUNK >> 4) + 2 * u, b_d + c * (CHUNK >> 4) + 2 * u, id_s, (c | u) != 0);
                mma_commit(&sh.s_full[t]);
            };
            const auto products = [&](uint32_t g, int t, int j) {
                const uint32_t a_d = tmem + S_COL + t * 128, d = tmem + O_COL + t * 128;
                const uint64_t b_d = vd + (g & 1) * (Z::TILE * (CHUNK >> 4));
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    mma_ts(d, a_d + 8 * u, b_d + u * (2048 >> 4), id_o, (j | u) != 0);
            };
            // the tile's number through all items, and the numbers of tiles, items and cleared
            // tails so far, as far as parities go
            uint32_t g = 0, q_uses[2] = {0, 0}, p_uses[2] = {0, 0}, tails = 0;
            for (uint32_t item = 0;; ++item) {
                const Item my = sh.item[item & 1];
                const Extent x(p, my);
                const int last = x.last();
                if (x.n > 0) {
                    if (!wait(sh, &sh.k_full[g & 1], (g >> 1) & 1)) break;
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        if (x.tiles(t) > 0) {
                            if (!wait(sh, &sh.q_full[t], q_uses[t] & 1)) break;
                            ++q_uses[t];
                            tc_fence_after();
                            scores(g, t);
                            if (x.tiles(t) == 1) mma_commit(&sh.q_free[t]);
                        }
                    mma_commit(&sh.k_free[g & 1]);
                }
                for (int j = 0; j < x.n && !sh.abort; ++j, ++g) {
                    if (!wait(sh, &sh.v_full[g & 1], (g >> 1) & 1)) break;
                    bool keys = false;  // tile j + 1's have been waited for
                    if (j == x.tail && !wait(sh, &sh.v_clean, tails++ & 1)) break;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int nt = x.tiles(t);
                        if (j >= nt) continue;
                        if (!wait(sh, &sh.p_ready[t], p_uses[t]++ & 1)) break;
                        tc_fence_after();
                        products(g, t, j);
                        if (t == last) mma_commit(&sh.v_free[g & 1]);
                        if (j + 1 == nt) mma_commit(&sh.o_done[t]);
                        if (j + 1 < nt) {
                            if (!keys && !wait(sh, &sh.k_full[(g + 1) & 1], ((g + 1) >> 1) & 1)) break;
                            keys = true;
                            scores(g + 1, t);
                            if (j + 2 == nt) mma_commit(&sh.q_free[t]);
                            if (t == last) mma_commit(&sh.k_free[(g + 1) & 1]);
                        }
                    }
                }
                mbar_arrive(&sh.item_free[item & 1]);
                if (sh.abort || !next_item(item)) break;
            }
            mma_commit(&sh.drained);
            wait_out(&sh.drained, 0);
        }
    } else if (warp == 2) {
        // ---- the items after the first, each as soon as the one two before it is left behind
        Item it = sh.item[0];
        for (uint32_t item = 0;; ++item) {
            const Extent was(p, it);
            it.g0 += was.n;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                it.met[t] += was.tiles(t);
                it.outputs[t] += was.tiles(t) > 0;
            }
            const bool more = next(it);
            if (!more) it.head = -1;
            if (!__all_sync(0xFFFFFFFFu, item == 0 || wait_far(sh, &sh.item_free[(item - 1) & 1],
                                                               ((item - 1) >> 1) & 1)))
                break;
            if (lane == 0) {
                sh.item[(item + 1) & 1] = it;
                mbar_arrive(&sh.item_full[(item + 1) & 1]);
            }
            __syncwarp();
            if (!more) break;
        }
    }
    if (warp == 2 && lane == 0 && !cut_here) p.plan[blockIdx.x] = make_int4(0, 0, 0, 0);
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
        pdl_launch_dependents();
        if (sh.abort && p.status) atomicOr(p.status, MTPSPEC_STATUS_TIMEOUT);
    }
    if (warp == 3) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(TMEM_COLS)
                     : "memory");
    }
}

// Units cut among CTAs: each row's partial outputs, weighted by their sums, become the output.  A
// warp a row; blockIdx.y is the CTA of the first kernel in which the unit starts.
constexpr int JOIN_THREADS = 256, JOIN_WARPS = JOIN_THREADS / 32;

template <typename T, int NC>
__global__ void __launch_bounds__(JOIN_THREADS) k_heads_join(const Params p) {
    pdl_wait_primary();
    const int4 u = p.plan[blockIdx.y];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rr = blockIdx.x * JOIN_WARPS + warp, r = rr % TM;
    const int tok_in = r / p.G, tok = rr / TM * p.TOK + tok_in;
    // (what an aborted call left there is checked)
    if (u.w < 2 || u.w > GRID - static_cast<int>(blockIdx.y) || u.x < 0 || u.y < 0 || u.x + u.y > p.Tq ||
        u.z < 0 || u.z >= p.Hkv || tok_in >= p.TOK || tok >= u.y)
        return;
    const int h = u.z * p.G + r - tok_in * p.G;
    // a CTA's partial of this row: the second slot where the unit starts, else the first
    const auto part_row = [&](int i) {
        return static_cast<int64_t>(2 * (blockIdx.y + i) + (i == 0)) * (2 * TM) + rr;
    };
    float top = -INFINITY, sum = 0.0f;
    for (int i = lane; i < u.w; i += 32) top = fmaxf(top, p.part_lse[part_row(i)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const float ref = top == -INFINITY ? 0.0f : top;
    constexpr int PER = 2 * NC;  // a lane's columns
    float acc[PER] = {};
#pragma unroll 4
    for (int i = 0; i < u.w; ++i) {
        const int64_t row = part_row(i);
        const float w = exp2f(p.part_lse[row] - ref);
        sum += w;
        float v[PER];
#pragma unroll
        for (int k = 0; k < PER; k += 2)
            *reinterpret_cast<float2 *>(v + k) =
                *reinterpret_cast<const float2 *>(p.part + row * (64 * NC) + k * 32 + lane * 2);
#pragma unroll
        for (int k = 0; k < PER; ++k) acc[k] += w * v[k];
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int64_t out_row = u.x + tok;
    uint16_t *dst = p.out + out_row * p.out_tok + h * p.out_head;
#pragma unroll
    for (int k = 0; k < PER; k += 2)
        if (k * 32 + lane * 2 < p.D)
            *reinterpret_cast<uint32_t *>(dst + k * 32 + lane * 2) = T::narrow2(acc[k] * inv, acc[k + 1] * inv);
    if (p.lse && lane == 0) p.lse[out_row * p.Hq + h] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * LN2;
}

struct Layout {
    size_t plan, part, lse, total;
};
Layout layout(int32_t D) {
    const auto align256 = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
    Layout y;
    y.plan = 0;
    y.part = align256(GRID * sizeof(int4));
    y.lse = y.part + static_cast<size_t>(2 * GRID) * 2 * TM * ((D + 63) / 64 * 64) * 4;
    y.total = y.lse + align256(static_cast<size_t>(2 * GRID) * 2 * TM * 4);
    return y;
}

template <typename T, int NC>
cudaError_t launch(const Maps &maps, const Params &p, cudaStream_t stream) {
    constexpr int smem = Sizes<NC>::SMEM;
    static AttrCache attr;
    cudaError_t e = ensure_attr(k_heads_chunk<T, NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem, attr);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(GRID);
    cfg.blockDim = dim3(NTHREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = pdl_attr();  // set up beside the end of whatever the stream runs before
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_heads_chunk<T, NC>, maps, p);
    if (e != cudaSuccess) return e;
    count_launches(1);
    cfg.gridDim = dim3(2 * TM / JOIN_WARPS, GRID);
    cfg.blockDim = dim3(JOIN_THREADS);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, k_heads_join<T, NC>, p);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

template <typename T>
cudaError_t pick(const Maps &maps, const Params &p, cudaStream_t stream) {
    return p.D <= 64 ? launch<T, 1>(maps, p, stream) : launch<T, 2>(maps, p, stream);
}

}  // namespace hch

size_t heads_chunk_workspace_bytes(int32_t D) { return hch::layout(D).total; }

cudaError_t run_heads_chunk(const HeadsAttnArgs &a, int dtype, cudaStream_t stream) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    hch::Params p = {};
    p.G = a.Hq / a.Hkv;
    p.TOK = hch::TM / p.G;
    // boxes of the largest power of two (up to a tile) that divides the page: a box never leaves
    // its page, and its rows start at a multiple of eight, the swizzle's period
    p.box_rows = std::min(hch::TN, a.page_size & -a.page_size);
    // an axis of one element may come with any stride
    const int64_t slot = a.slot_stride, head = a.Hkv == 1 ? a.D : a.head_stride;
    const int64_t page = a.num_pages == 1 ? slot * a.page_size : a.page_stride;
    const int64_t q_head = a.Hq == 1 ? a.D : a.q_head, q_tok = a.Tq == 1 ? a.D : a.q_tok;
    const auto encode = [&](CUtensorMap *m, const uint16_t *ptr, const cuuint64_t (&dims)[4],
                            const cuuint64_t (&strides)[3], const cuuint32_t (&box)[4]) {
        const cuuint32_t es[4] = {1, 1, 1, 1};
        return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t *>(ptr), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    const auto u = [](int64_t x) { return static_cast<cuuint64_t>(x); };
    hch::Maps maps;
    const cuuint64_t qd[4] = {u(a.D), u(p.G), u(a.Tq), u(a.Hkv)}, qs[3] = {u(q_head * 2), u(q_tok * 2), u(q_head * p.G * 2)};
    const cuuint64_t cd[4] = {u(a.D), u(a.Hkv), u(a.page_size), u(a.num_pages)}, cs[3] = {u(head * 2), u(slot * 2), u(page * 2)};
    const cuuint32_t qb[4] = {64, static_cast<cuuint32_t>(p.G), static_cast<cuuint32_t>(p.TOK), 1};
    const cuuint32_t cb[4] = {64, 1, static_cast<cuuint32_t>(p.box_rows), 1};
    if (!encode(&maps.q, a.q, qd, qs, qb) || !encode(&maps.k, a.k_cache, cd, cs, cb) ||
        !encode(&maps.v, a.v_cache, cd, cs, cb))
        return cudaErrorInvalidValue;
    const hch::Layout y = hch::layout(a.D);
    unsigned char *ws = static_cast<unsigned char *>(a.workspace);
    p.cu_q = a.cu_q;
    p.kv_len = a.kv_len;
    p.block_table = a.block_table;
    p.max_pages = a.max_pages;
    p.max_len = static_cast<int>(std::min<int64_t>(a.max_pages * a.page_size, (int64_t{1} << 31) - 256));
    p.num_pages = static_cast<int>(a.num_pages);
    p.page_size = a.page_size;
    p.B = static_cast<int>(a.B);
    p.Tq = static_cast<int>(a.Tq);
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.D = a.D;
    p.window = a.window;
    p.sinks = a.sinks;
    p.scale2 = a.scale * hch::LOG2E;
    p.out = a.out;
    p.out_tok = a.out_tok;
    p.out_head = a.out_head;
    p.lse = a.lse;
    p.plan = reinterpret_cast<int4 *>(ws + y.plan);
    p.part = reinterpret_cast<float *>(ws + y.part);
    p.part_lse = reinterpret_cast<float *>(ws + y.lse);
    p.status = a.status;
    return dtype == MTPSPEC_BF16 ? hch::pick<Bf16>(maps, p, stream) : hch::pick<F16>(maps, p, stream);
}

}  // namespace mtpspec
