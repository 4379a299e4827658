// Attention with grouped heads over the paged cache: draft steps, verifications, chunks of prompts and
// whole prompts, in any mix.
//
// One pass over the keys with the running maximum m and sum l of a softmax: for a tile of keys
//     S = Q K^T,  p = 2^(s - m),  l += sum p,  O += p V,  and O, l scaled by 2^(m - m') when m
// changes (s, m in powers of two, scale * log2 e folded in; m follows a row's maximum only when
// that has grown by more than 2^8).  Weights are rounded to 16 bits for the second product; l
// sums the unrounded ones in fp32.  (In fp16 m lies 2^7 below that maximum, so that fewer weights
// are subnormal: half_types.cuh.)
//
// Rows: the G = Hq / Hkv query heads of a key head meet the same keys, so a unit's 128 rows are
// 128 / G tokens times G heads, two threads a row in the softmax.  (Four threads a row: 313 -> 349 us
// in the second case below.)
//
// Keys: tiles of 128, or of 64 for heads of more than 128 elements.  Tensor memory holds the output
// and two score buffers, whose first halves become the weights (the left operand of the second
// product): the tensor cores compute the scores two tiles ahead, so that a softmax waits for little
// but the softmax before.  (Two row tiles of one buffer each beside two outputs: 340 us in that case; a
// round took what the chain scores - softmax - products of a row tile takes, 4,100 cycles for 2,300
// of products.)  Keys and values have a ring of tiles each.
//
// A tile is brought in boxes that stay within a page; a copy takes the thread that issues it some 75
// cycles, so there are four such threads.  With a window, a unit meets the tiles of the first tokens,
// then those of the window.
//
// Work: all units laid end to end, a unit's length its key tiles and a constant for its start and
// end, and cut evenly over 152 CTAs, one a multiprocessor, whatever the lengths; every CTA finds
// its start from a scan of the rows.  A unit cut among CTAs leaves fp32 partial outputs, which a
// second small kernel joins.
//
// What bounds it (HBM copy 6.8 TB/s, products 1885 TFLOP/s measured; in a graph):
//   8 prompts of 77-1500 tokens, 32 / 4 heads of 128, pages of 16, bf16, 66 GFLOP: 93 us, 0.71 PFLOP/s.
//     Units have six tiles on average, and nothing covers their starts and ends, which weigh as much
//     as some three tiles (tensor pipe 31 %).
//   6 rows of 1-1000 tokens behind up to 7001 keys, 40 / 8 heads of 128, pages of 48, fp16, 365 GFLOP:
//     300 us, 1.22 PFLOP/s, 0.64 (at 2070 MHz; in a long run the power limit leaves some 1800, and it is 322
//     us).  A tile takes some 1,900 cycles, and the softmax of its 128 x 128 scores by eight warps is the
//     longest part (tensor pipe 55 %, issue slots 47 %, 2^x pipe 29 %).
//   256 rows of 4 tokens over 500-4000 keys, 32 / 8 heads of 128, pages of 64, bf16, 2.39 GB: 377 us, 6.3
//     TB/s, 0.93 of the copy rate.
//   8192 tokens, 16 / 2 heads of 256, pages of 128, bf16, 550 GFLOP: 461 us, 1.19 PFLOP/s, 0.63.  Tiles
//     are half as long, as two of 128 keys of such heads do not fit (tensor pipe 50 %, the products'
//     reads of shared memory 50 %, issue slots 30 %).
#include <algorithm>

#include "heads.cuh"

namespace mtpspec {
namespace hch {

using namespace heads;

constexpr int TM = 128;            // rows of a unit
constexpr int Q_CHUNK = TM * 128;  // bytes of a unit's rows x 64 columns of 16 bits
constexpr int THREADS = 448;       // warps 0, 3, 12, 13 TMA, 1 MMA, 2 items; 4-11 softmax
constexpr uint32_t TMEM_COLS = 512;
constexpr int O_COL = 256;         // the output; the score buffers lie at 0 and 128
constexpr int AHEAD = 2;           // key tiles that the scores are ahead of the products
constexpr int ITEMS = 4;
constexpr int MAX_SLOTS = 4;       // tiles of either ring

// An item of a CTA: tiles i0 .. i1 - 1 of a unit's list of n.  Its `tiles` are at least one.  head -1:
// no more.
template <int TN>
struct Item {
    Unit<TN> u;
    int row, head, i0, i1, n, tiles;
};

// Barriers by tile are doubled, a phase for every other tile: who waits for a tile may be one behind,
// and a parity cannot tell two phases from none.
template <int TN>
struct __align__(16) Shared {
    uint64_t k_full[MAX_SLOTS], k_free[MAX_SLOTS], v_full[MAX_SLOTS], v_free[MAX_SLOTS];
    uint64_t q_full[2], q_free[2], s_full[2], p_ready[2], pv_done[2], drained;
    uint64_t item_full[ITEMS], item_free[ITEMS];
    Item<TN> item[ITEMS];
    uint32_t tmem;
    volatile int abort;
    int2 box[4][8];         // boxes of a tile, by producer
    float other[2][2][TM];  // what the two threads of a row tell each other, in turn, by half
};

// NC: the 64-column chunks of a head.
template <int NC>
struct Sizes {
    static constexpr int TN = NC <= 2 ? 128 : 64;          // keys of a tile
    static constexpr int CHUNK = TN * 128, TILE = NC * CHUNK;
    static constexpr int QS = NC <= 2 ? 2 : 1;             // units whose queries are there
    static constexpr int KS = NC == 1 ? 4 : 2, VS = NC == 1 ? 4 : 3;  // tiles of the keys' and the values' ring
    static constexpr int Q_BYTES = NC * Q_CHUNK;
    static constexpr int EXTRA = static_cast<int>(sizeof(Shared<TN>));
    static constexpr int SMEM = QS * Q_BYTES + (KS + VS) * TILE + EXTRA;
    static_assert(SMEM <= 232448, "227 KB a CTA");
    static_assert(SMEM > 116 * 1024, "two CTAs, which take all tensor memory, may not share an SM");
};

template <typename T, int NC>
__global__ void __launch_bounds__(THREADS, 1)
k_heads_chunk(const __grid_constant__ Maps maps, const Params p) {
    extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle's period
    using Z = Sizes<NC>;
    constexpr int TN = Z::TN, C = TN / 2, CHUNK = Z::CHUNK, TILE = Z::TILE, KS = Z::KS, VS = Z::VS, QS = Z::QS;
    using Item = hch::Item<TN>;
    const uint32_t q_s = smem_addr(smem), k_s = q_s + QS * Z::Q_BYTES, v_s = k_s + KS * TILE;
    Shared<TN> &sh = *reinterpret_cast<Shared<TN> *>(smem + Z::SMEM - Z::EXTRA);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < MAX_SLOTS; ++i) {
            mbar_init(&sh.k_full[i], 1);
            mbar_init(&sh.k_free[i], 1);
            mbar_init(&sh.v_full[i], 1);
            mbar_init(&sh.v_free[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.q_full[i], 1);
            mbar_init(&sh.q_free[i], 1);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_ready[i], 8);
            mbar_init(&sh.pv_done[i], 1);
        }
        for (int i = 0; i < ITEMS; ++i) {
            mbar_init(&sh.item_full[i], 1);
            mbar_init(&sh.item_free[i], 13);  // the producers, the issuer, eight softmax warps
        }
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
    // ---- where this CTA starts, and its first item
    Walk<TN> walk;
    const Cut cut = find_start<TN, THREADS>(p, *reinterpret_cast<Scan *>(smem), 2, walk);  // (before any copy)
    // the next item with tiles to meet; a unit that sees no key is done with at once
    const auto next = [&](Item &it) {
        it.head = -1;
        while (walk.next(p, cut, it.u, it.i0, it.i1, it.n)) {
            it.tiles = min(it.i1, it.u.tiles(p)) - it.i0;
            if (it.tiles > 0) {
                it.row = walk.row;
                it.head = walk.head;
                return;
            }
            const int rows = min(TM, it.u.nq * p.G - it.u.m0);
            for (int r = 0; r < min(rows, p.unit_rows); ++r) {
                const int m = it.u.m0 + r, tok = m / p.G, h = walk.head * p.G + m - tok * p.G;
                uint16_t *dst = p.out + (it.u.q0 + tok) * p.out_tok + h * p.out_head;
                for (int d = lane * 8; d < p.D; d += 256) *reinterpret_cast<uint4 *>(dst + d) = make_uint4(0, 0, 0, 0);
                if (lane == 0 && p.lse) p.lse[static_cast<int64_t>(it.u.q0 + tok) * p.Hq + h] = -INFINITY;
            }
        }
    };
    if (warp == 2) {
        Item it = {};
        next(it);
        if (lane == 0) {
            sh.item[0] = it;
            mbar_arrive(&sh.item_full[0]);
        }
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    // Every role goes through the CTA's items: is there one of number `item`, and no abort?
    const auto there_is = [&](uint32_t item) {
        return wait_far(sh, &sh.item_full[item % ITEMS], (item / ITEMS) & 1) && sh.item[item % ITEMS].head >= 0;
    };

    if (warp >= 4 && warp < 12) {
        // ---- softmax: two threads a row, half of a tile's keys each
        const int half = (warp - 4) >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lane_bits = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t o_t = tmem + lane_bits + O_COL;
        const int my_tok = r / p.G, last_tok = p.unit_rows / p.G - 1;  // within the unit
        const int pair_bar = 1 + (warp & 3);
        int turn = 0;
        // the row's value from those of its threads
        const auto meet = [&](float v, auto join) {
            sh.other[turn][half][r] = v;
            asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory");
            v = join(v, sh.other[turn][half ^ 1][r]);
            turn ^= 1;
            return v;
        };
        uint32_t g = 0;  // the tile's number
        for (uint32_t item = 0; all_say<64>(there_is(item), pair_bar); ++item) {
            // (what only the item's end needs stays in shared memory meanwhile)
            const volatile Item &my = sh.item[item % ITEMS];
            const int tiles = my.tiles, len = my.u.len, ns = my.u.ns, skip = my.u.w0 - ns, i0 = my.i0;
            // the tile that the row's keys end in, if that is not a whole one
            const int tail = (len % TN != 0 ? ns + len / TN - my.u.w0 : -1) - i0;
            const int tok = my.u.m0 / p.G + my_tok;
            const int limit = len - my.u.nq + tok + 1;  // one past the last key that this row sees,
            const int sure = limit - my_tok;            // and the least of the unit's rows
            const int width = p.window > 0 && p.window < len ? p.window : 0;
            float m_ref = -INFINITY, l = 0.0f;
            for (int j = 0; j < tiles; ++j, ++g) {
                const uint32_t b = g & 1, s_b = tmem + lane_bits + b * TN;
                wait_long(sh, &sh.s_full[b], (g >> 1) & 1);
                tc_fence_after();
                uint32_t x[C / 32][32];
#pragma unroll
                for (int c = 0; c < C / 32; ++c) tmem_ld32(s_b + half * C + 32 * c, x[c]);
                if (__builtin_expect(j == tail, 0)) {
                    // value rows behind the row's last key: whatever lies there must not meet the
                    // zero weights
                    const int z0 = len % TN;
                    const uint32_t slot = g % VS;
                    wait(sh, &sh.v_full[slot], (g / VS) & 1);
#pragma unroll 1
                    for (int c = 0; c < NC; ++c) {
                        const uint32_t v = v_s + slot * TILE + c * CHUNK + z0 * 128;
#pragma unroll 1
                        for (int i = half * 128 + r; i < (TN - z0) * 8; i += 256)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(v + i * 16), "r"(0)
                                         : "memory");
                    }
                    fence_async_smem();
                }
                tmem_wait_ld();
                const int key0 = (i0 + j < ns ? i0 + j : i0 + j + skip) * TN;
                if (__builtin_expect(key0 + TN > sure, 0)) {  // more than every row sees
                    const int seen = limit - key0 - half * C;
#pragma unroll
                    for (int i = 0; i < C; ++i)
                        if (i >= seen) x[i / 32][i % 32] = 0xFF800000u;
                }
                if (__builtin_expect(width && key0 < sure + last_tok - width, 0)) {  // not in every window
                    const int first = max(p.sinks - key0, 0) - half * C;
                    const uint32_t gap = max(limit - width - key0 - half * C - first, 0);  // hidden from `first` on
#pragma unroll
                    for (int i = 0; i < C; ++i)
                        if (static_cast<uint32_t>(i - first) < gap) x[i / 32][i % 32] = 0xFF800000u;
                }
                float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < C; i += 2)
                    top4[(i >> 1) & 3] = max3(top4[(i >> 1) & 3], __uint_as_float(x[i / 32][i % 32]),
                                              __uint_as_float(x[i / 32][i % 32 + 1]));
                const float top = meet(fmaxf(max3(top4[0], top4[1], top4[2]), top4[3]),
                                       [](float a, float b) { return fmaxf(a, b); }) * p.scale2;
                const bool raise = top > m_ref + (LAZY + T::first_weight);
                const float m_new = top - T::first_weight;
                if (__builtin_expect(j > 0 && __any_sync(0xFFFFFFFFu, raise), 0)) {
                    wait(sh, &sh.pv_done[b ^ 1], ((g - 1) >> 1) & 1);  // the output is free
                    tc_fence_after();
                    const float f = raise ? ex2(m_ref - m_new) : 1.0f;
                    l *= f;
#pragma unroll 1
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
                for (int c = 0; c < C / 32; ++c) {
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
                    // (both threads of the row have read their scores: they have met since)
                    tmem_st16(s_b + half * (C / 2) + 16 * c, w);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_ready[b]);
                float l0, l1;
                unpack2(add2(part[0], part[1]), l0, l1);
                l += l0 + l1;
            }
            l = meet(l, [](float a, float b) { return a + b; });
            wait_long(sh, &sh.pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1);
            tc_fence_after();
            // (a sum of zero: nothing was seen; one that is NaN stays so)
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const float lse2 = l == 0.0f ? -INFINITY : m_ref + log2f(l);
            const int h = my.head * p.G + r - my_tok * p.G;
            const bool real = r < p.unit_rows && tok < my.u.nq;
            const bool whole = i0 == 0 && my.i1 == my.n;
            const int64_t out_row = my.u.q0 + tok;
            const int slot_out = 2 * blockIdx.x + (i0 > 0 ? 0 : 1);
            if (real && half == 0) {
                if (!whole)
                    p.part_lse[static_cast<int64_t>(slot_out) * TM + r] = lse2;
                else if (p.lse)
                    p.lse[out_row * p.Hq + h] = lse2 * LN2;
            }
            uint16_t *dst = p.out + out_row * p.out_tok + h * p.out_head;
            // 32 bytes a store, a whole sector, where the rows allow it
            const bool sectors = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;
#pragma unroll 1
            for (int col = half * (NC * 32); col < (half + 1) * (NC * 32); col += 32) {
                uint32_t o[32];
                __syncwarp();
                tmem_ld32(o_t + col, o);
                tmem_wait_ld();
                if (!real) continue;
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        *part_at<NC, TM>(p, slot_out, col + i, r) =
                            make_float4(__uint_as_float(o[i]), __uint_as_float(o[i + 1]),
                                        __uint_as_float(o[i + 2]), __uint_as_float(o[i + 3]));
                    continue;
                }
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    if (col + v * 16 >= p.D) break;
                    uint32_t y[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        y[u] = T::narrow2(__uint_as_float(o[16 * v + 2 * u]), __uint_as_float(o[16 * v + 2 * u + 1]));
                    uint16_t *d = dst + col + v * 16;
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
            if (lane == 0) mbar_arrive(&sh.item_free[item % ITEMS]);
        }
    } else if (warp == 0 || warp == 3 || warp >= 12) {
        // ---- producers: two of the keys and two of the values, half of a tile's boxes each (a copy takes
        // a thread some 75 cycles, and a tile of 128 keys in pages of 16 is 16 of them for its keys
        // alone).  A lane finds a box, and one thread issues.
        const int what = warp == 3 || warp == 13, part = warp >= 12;  // values or keys; which boxes
        const int boxes = TN / p.box_rows, mine = part ? boxes / 2 : (boxes + 1) / 2, first = part ? (boxes + 1) / 2 : 0;
        const auto all = [](bool yes) { return __all_sync(0xFFFFFFFFu, yes) != 0; };
        const uint32_t N = what ? VS : KS, ring = what ? v_s : k_s;
        const CUtensorMap *map = what ? &maps.v : &maps.k;
        uint64_t *full = what ? sh.v_full : sh.k_full, *free = what ? sh.v_free : sh.k_free;
        int2 *at = sh.box[what * 2 + part];
        uint32_t slot = 0, phase = 1, fills = 0, q_uses = 0;
        bool ok = true;
        for (uint32_t item = 0; ok && all(there_is(item)); ++item) {
            const Item &my = sh.item[item % ITEMS];
            const int32_t *table = p.block_table + static_cast<int64_t>(my.row) * p.max_pages;
            const int tiles = my.tiles, i0 = my.i0, head = my.head, len = my.u.len, ns = my.u.ns, skip = my.u.w0 - ns;
            const int q_tok = my.u.q0 + my.u.m0 / p.G, window = my.u.window(p);
            Box box = {};  // of the next tile
            const auto look = [&](int i) {
                const int key = (i0 + i < ns ? i0 + i : i0 + i + skip) * TN;
                box.look(p, table, key + (first + lane) * p.box_rows, len, window, lane < mine);
            };
            look(0);
            for (int i = 0; ok && i < tiles; ++i) {
                if (lane < mine) at[lane] = box.settle(p);
                if (i + 1 < tiles) look(i + 1);
                __syncwarp();
                if (elect_one()) {
                    ok = wait(sh, &free[slot], phase);
                    if (ok) {
                        if (part == 0) mbar_expect_tx(&full[slot], TILE);
                        const uint32_t dst = ring + slot * TILE + first * p.box_rows * 128;
#pragma unroll 4
                        for (int x = 0; x < mine; ++x) {
                            const int2 to = at[x];
#pragma unroll
                            for (int c = 0; c < NC; ++c)
                                tma_load_4d(dst + c * CHUNK + x * p.box_rows * 128, map, c * 64, to.y, head, to.x, &full[slot]);
                        }
                    }
                    if (ok && i == 0 && what == 0 && part == 0) {  // the queries, behind the first keys, which wait for less
                        const uint32_t s = item % QS;
                        ok = wait_long(sh, &sh.q_free[s], (item / QS + 1) & 1);
                        if (ok) {
                            mbar_expect_tx(&sh.q_full[s], NC * p.unit_rows * 128);
                            for (int c = 0; c < NC; ++c)
                                tma_load_4d(q_s + s * Z::Q_BYTES + c * Q_CHUNK, &maps.q, c * 64, 0, q_tok, head,
                                            &sh.q_full[s]);
                        }
                    }
                }
                __syncwarp();
                ok = all(ok);
                ++fills;
                if (++slot == N) {
                    slot = 0;
                    phase ^= 1;
                }
            }
            ++q_uses;
            __syncwarp();  // (all lanes have read the item)
            if (lane == 0) mbar_arrive(&sh.item_free[item % ITEMS]);
        }
        if (__any_sync(0xFFFFFFFFu, sh.abort)) {
            // let the copies in flight land: the last fill of every slot, and the queries' (a fill that
            // was cut off never completes: its wait runs to the limit)
            for (uint32_t s = 0; s < N; ++s)
                if (fills > s) wait_out(&full[s], ((fills + N - 1 - s) / N - 1) & 1);
            for (uint32_t s = 0; s < QS; ++s)
                if (what == 0 && part == 0 && q_uses > s) wait_out(&sh.q_full[s], ((q_uses + QS - 1 - s) / QS - 1) & 1);
        }
    } else if (warp == 1) {
        if (elect_one()) {
            // ---- MMA issuer: a tile's products, then the scores of the tile two on
            constexpr uint32_t id_s = idesc_of<T>(TM, TN, false), id_o = idesc_of<T>(TM, 64 * NC, true);
            const uint64_t qd = smem_desc_sw128(q_s), kd = smem_desc_sw128(k_s), vd = smem_desc_rows_k(v_s, CHUNK);
            uint32_t gk = 0, gv = 0;  // the numbers of the next tiles
            for (uint32_t item = 0; there_is(item); ++item) {
                const int tiles = sh.item[item % ITEMS].tiles;
                const uint32_t q = item % QS;
                if (!wait(sh, &sh.q_full[q], (item / QS) & 1)) break;
                for (int j = -AHEAD; j < tiles && !sh.abort; ++j) {
                    if (j >= 0) {
                        const uint32_t b = gv & 1, slot = gv % VS;
                        if (!wait(sh, &sh.v_full[slot], (gv / VS) & 1)) break;
                        if (!wait(sh, &sh.p_ready[b], (gv >> 1) & 1)) break;
                        tc_fence_after();
                        const uint64_t b_d = vd + slot * (TILE >> 4);
#pragma unroll
                        for (int u = 0; u < TN / 16; ++u)
                            mma_ts(tmem + O_COL, tmem + b * TN + 8 * u, b_d + u * (2048 >> 4), id_o, (j | u) != 0);
                        mma_commit(&sh.pv_done[b]);
                        mma_commit(&sh.v_free[slot]);
                        ++gv;
                    }
                    if (j + AHEAD < tiles) {
                        const uint32_t b = gk & 1, slot = gk % KS;
                        if (!wait(sh, &sh.k_full[slot], (gk / KS) & 1)) break;
                        const uint64_t a_d = qd + q * (Z::Q_BYTES >> 4), b_d = kd + slot * (TILE >> 4);
#pragma unroll
                        for (int c = 0; c < NC; ++c)
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                mma_bf16(tmem + b * TN, a_d + c * (Q_CHUNK >> 4) + 2 * u, b_d + c * (CHUNK >> 4) + 2 * u, id_s,
                                         (c | u) != 0);
                        mma_commit(&sh.s_full[b]);
                        mma_commit(&sh.k_free[slot]);
                        if (j + AHEAD + 1 == tiles) mma_commit(&sh.q_free[q]);
                        ++gk;
                    }
                }
                mbar_arrive(&sh.item_free[item % ITEMS]);
                if (sh.abort) break;
            }
            mma_commit(&sh.drained);
            wait_out(&sh.drained, 0);
        }
    } else if (warp == 2) {
        // ---- the items after the first, each as soon as its place is left behind
        Item it = sh.item[0];
        for (uint32_t item = 1; it.head >= 0; ++item) {
            next(it);
            if (!__all_sync(0xFFFFFFFFu, item < ITEMS || wait_far(sh, &sh.item_free[item % ITEMS],
                                                                  (item / ITEMS - 1) & 1)))
                break;
            if (lane == 0) {
                sh.item[item % ITEMS] = it;
                mbar_arrive(&sh.item_full[item % ITEMS]);
            }
            __syncwarp();
        }
        walk.close(p);
    }
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

struct Layout {
    size_t plan, part, lse, total;
};
Layout layout(int NC) {
    const auto align256 = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
    const size_t rows = static_cast<size_t>(2 * SMS) * TM;
    Layout y;
    y.plan = 0;
    y.part = align256(SMS * sizeof(Plan));
    y.lse = y.part + rows * (64 * NC) * 4;
    y.total = y.lse + align256(rows * 4);
    return y;
}

template <typename T, int NC>
cudaError_t launch(const HeadsAttnArgs &a, cudaStream_t stream) {
    using Z = Sizes<NC>;
    const Layout y = layout(NC);
    const int G = a.Hq / a.Hkv;
    Params p;
    Maps maps;
    if (!set_up(a, TM / G * G, Z::TN, true, y.plan, y.part, y.lse, p, maps)) return cudaErrorInvalidValue;
    static AttrCache attr;
    cudaError_t e = ensure_attr(k_heads_chunk<T, NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, Z::SMEM, attr);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(SMS);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = Z::SMEM;
    cfg.stream = stream;
    cfg.attrs = pdl_attr();  // set up beside the end of whatever the stream runs before
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_heads_chunk<T, NC>, maps, p);
    if (e != cudaSuccess) return e;
    count_launches(1);
    return launch_join<T, NC, TM>(cfg, p, stream);
}
template <typename T>
cudaError_t pick(const HeadsAttnArgs &a, cudaStream_t s) {
    return a.D <= 64 ? launch<T, 1>(a, s) : a.D <= 128 ? launch<T, 2>(a, s) : launch<T, 4>(a, s);
}

}  // namespace hch

size_t heads_chunk_workspace_bytes(int32_t D) { return hch::layout(D <= 64 ? 1 : D <= 128 ? 2 : 4).total; }

cudaError_t run_heads_chunk(const HeadsAttnArgs &a, int dtype, cudaStream_t stream) {
    return dtype == MTPSPEC_BF16 ? hch::pick<Bf16>(a, stream) : hch::pick<F16>(a, stream);
}

}  // namespace mtpspec
