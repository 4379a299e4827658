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
// 128 / G tokens times G heads.  A unit of work is two such tiles (one, for heads of more than 128
// elements), a thread a row in the softmax.
//
// Keys: tiles of 128, and a score buffer a row tile, whose first half becomes the weights (the left
// operand of the second product): while the tensor cores work on one row tile, the other's softmax
// runs.  A single row tile has two buffers, of 64 keys, beside its 256 output columns: the scores of
// a tile are there before the weights of the one before are.
//
// A tile is brought in boxes that stay within a page, a box a lane of the producing warp.  With a
// window, a unit meets the tiles of the first tokens, then those of the window.
//
// Work: all units laid end to end, a unit's length its key tiles and a constant for its start and
// end, and cut evenly over 152 CTAs, one a multiprocessor, whatever the lengths; every CTA finds
// its start from a scan of the rows.  A unit cut among CTAs leaves fp32 partial outputs, which a
// second small kernel joins.
#include <algorithm>

#include "heads.cuh"

namespace mtpspec {
namespace hch {

using namespace heads;

constexpr int TM = 128;            // rows of a tile in tensor memory
constexpr int Q_CHUNK = TM * 128;  // bytes of a row tile x 64 columns of 16 bits
constexpr uint32_t TMEM_COLS = 512;
constexpr int O_COL = 256;         // row tile t's scores: 128 t, its output: 256 + 128 t
constexpr int ITEMS = 4;

// An item of a CTA: tiles i0 .. i1 - 1 of a unit's list of n (at least 1); how many of them either
// row tile meets, and which of them the row's keys end in, if that is not a whole tile; with the key
// tiles before it, and the key tiles that either row tile met before.  head -1: no more.
template <int TN>
struct Item {
    Unit<TN> u;
    int row, head, i0, i1, n;
    int nt[2], tail;
    uint32_t g0, met[2];
    __device__ __forceinline__ int tiles() const { return max(nt[0], nt[1]); }
};

constexpr int MAX_RING = 8;
// Barriers by row tile are doubled, a phase for every other key tile: who waits for a tile may be one
// behind, and a parity cannot tell two phases from none.
template <int TN>
struct __align__(16) Shared {
    uint64_t k_full[MAX_RING], v_full[MAX_RING], k_free[MAX_RING], v_free[MAX_RING];  // by the tile's slot
    uint64_t q_full[2], q_free[2], s_full[2][2], p_ready[2][2], pv_done[2][2], drained;
    uint64_t item_full[ITEMS], item_free[ITEMS];
    Item<TN> item[ITEMS];
    Scan scan;
    uint32_t tmem;
    volatile int abort;
    float other[2][2][TM];  // what the two threads of a row tell each other, by tile and half
};

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
// A tile whose rows are the products' K axis and whose 64-column chunks are `chunk` bytes apart.
__device__ __forceinline__ uint64_t smem_desc_rows_k(uint32_t addr, uint32_t chunk) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(chunk >> 4) << 16;
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

// NC: the 64-column chunks of a head.
template <int NC>
struct Sizes {
    static constexpr int NT = NC <= 2 ? 2 : 1;                      // row tiles of a unit
    static constexpr int TN = NC <= 2 ? 128 : 64;                   // keys of a tile
    static constexpr int SB = NC <= 2 ? 1 : 2;                      // score buffers of a row tile
    static constexpr int CHUNK = TN * 128;                          // bytes of a key tile x 64 columns
    static constexpr int HALVES = NT;                               // softmax threads of a row
    static constexpr int THREADS = 128 + 128 * NT * HALVES;         // warp 0 TMA, 1 MMA, 2 items, 3 TMEM; softmax
    static constexpr int TILE = 2 * NC * CHUNK, RING = 128 * 1024 / TILE;
    static constexpr int STAGE = 2048;                              // of a softmax warp: 32 rows x 32 columns
    static constexpr int Q_BYTES = NT * NC * Q_CHUNK, STAGES = Q_BYTES + RING * TILE;
    static constexpr int EXTRA = static_cast<int>(sizeof(Shared<TN>));
    static constexpr int SMEM = STAGES + (THREADS - 128) / 32 * STAGE + EXTRA;
    static_assert(SMEM <= 232448, "227 KB a CTA");
    static_assert(SMEM > 116 * 1024, "two CTAs, which take all tensor memory, may not share an SM");
};

template <typename T, int NC>
__global__ void __launch_bounds__(Sizes<NC>::THREADS, 1)
k_heads_chunk(const __grid_constant__ Maps maps, const Params p) {
    extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle's period
    using Z = Sizes<NC>;
    constexpr int NT = Z::NT, HALVES = Z::HALVES, TN = Z::TN, C = TN / HALVES, SB = Z::SB, CHUNK = Z::CHUNK, RING = Z::RING;
    using Item = hch::Item<TN>;
    const uint32_t q_s = smem_addr(smem), ring = q_s + Z::Q_BYTES;
    Shared<TN> &sh = *reinterpret_cast<Shared<TN> *>(smem + Z::SMEM - Z::EXTRA);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < RING; ++i) {
            mbar_init(&sh.k_full[i], 1);
            mbar_init(&sh.v_full[i], 1);
            mbar_init(&sh.k_free[i], 1);
            mbar_init(&sh.v_free[i], 1);
        }
        for (int t = 0; t < NT; ++t) {
            mbar_init(&sh.q_full[t], 1);
            mbar_init(&sh.q_free[t], 1);
            for (int b = 0; b < SB; ++b) {
                mbar_init(&sh.s_full[t][b], 1);
                mbar_init(&sh.p_ready[t][b], 4 * HALVES);
                mbar_init(&sh.pv_done[t][b], 1);
            }
        }
        for (int i = 0; i < ITEMS; ++i) {
            mbar_init(&sh.item_full[i], 1);
            mbar_init(&sh.item_free[i], 2 + 4 * NT * HALVES);  // the producer, the issuer, the softmax warps
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
    const Cut cut = find_start<TN, Z::THREADS>(p, sh.scan, 2, walk);
    const auto next = [&](Item &it) {
        const bool more = walk.next(p, cut, it.u, it.i0, it.i1, it.n);
        it.row = walk.row;
        it.head = more ? walk.head : -1;
        it.nt[0] = it.nt[1] = 0;
        if (more) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
                it.nt[t] = max(0, min(it.i1, it.u.tiles(p, it.u.m0 + t * p.tile_rows, p.tile_rows)) - it.i0);
            it.tail = it.u.tail() - it.i0;
        }
        return more;
    };
    if (warp == 2) {
        Item it = {};
        next(it);
        if (lane == 0) {
            sh.item[0] = it;
            mbar_arrive(&sh.item_full[0]);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    // Every role goes through the CTA's items: is there one of number `item`, and no abort?
    const auto there_is = [&](uint32_t item) {
        return wait_far(sh, &sh.item_full[item % ITEMS], (item / ITEMS) & 1) && sh.item[item % ITEMS].head >= 0;
    };

    if (warp >= 4) {
        // ---- softmax: a thread a row, or two, with 64 of a tile's 128 keys each
        const int t = (warp - 4) / (4 * HALVES), half = (warp - 4) / 4 % HALVES, r = (warp & 3) * 32 + lane;
        const uint32_t lane_bits = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_t = tmem + lane_bits + t * 128, o_t = tmem + lane_bits + O_COL + t * 128;
        const int my_tok = r / p.G, last_tok = p.tile_rows / p.G - 1;  // within the tile
        const int pair_bar = 1 + t * 4 + (warp & 3);
        // the row's value from those of its threads
        const auto meet = [&](float v, auto join) {
            if constexpr (HALVES == 2) {
                sh.other[t][half][r] = v;
                asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory");
                v = join(v, sh.other[t][half ^ 1][r]);
            }
            return v;
        };
        const auto go_on = [&](uint32_t item) {
            const bool yes = there_is(item);
            return HALVES == 2 ? both(yes, pair_bar) : yes;
        };
        for (uint32_t item = 0; go_on(item); ++item) {
            // (what only the item's end needs stays in shared memory meanwhile)
            const volatile Item &my = sh.item[item % ITEMS];
            const int nt = my.nt[t], len = my.u.len, ns = my.u.ns, skip = my.u.w0 - ns, i0 = my.i0;
            const int tail = my.tail;  // the tile whose values are to be cleared
            const int tok = (my.u.m0 + t * p.tile_rows) / p.G + my_tok;
            const int limit = len - my.u.nq + tok + 1;  // one past the last key that this row sees,
            const int sure = limit - my_tok;            // and the least of the tile's rows
            const int width = p.window > 0 && p.window < len ? p.window : 0;
            uint32_t met = my.met[t];  // the row tile's key tiles so far
            float m_ref = -INFINITY, l = 0.0f;
            for (int j = 0; j < nt; ++j, ++met) {
                const uint32_t buffer = met % SB, phase = (met / SB) & 1, s_b = s_t + buffer * TN;
                wait_long(sh, &sh.s_full[t][buffer], phase);
                tc_fence_after();
                uint32_t x[C / 32][32];
#pragma unroll
                for (int c = 0; c < C / 32; ++c) tmem_ld32(s_b + half * C + 32 * c, x[c]);
                if (__builtin_expect(j == tail, 0)) {
                    // value rows behind the row's last key: whatever lies there must not meet the
                    // zero weights.  (Either row tile clears them, before its own products.)
                    const uint32_t g = my.g0 + tail, slot = g % RING;
                    wait(sh, &sh.v_full[slot], (g / RING) & 1);
                    const int z0 = len % TN;
#pragma unroll 1
                    for (int c = 0; c < NC; ++c) {
                        const uint32_t v = ring + slot * Z::TILE + (NC + c) * CHUNK + z0 * 128;
#pragma unroll 1
                        for (int i = half * 128 + r; i < (TN - z0) * 8; i += 128 * HALVES)
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
                for (int i = 0; i < C / 2; ++i)
                    top4[i & 3] = max3(top4[i & 3], __uint_as_float(x[i / 32][i % 32]),
                                       __uint_as_float(x[C / 64 + i / 32][i % 32]));
                // (the second barrier of a tile is p_ready: nobody writes the next value before the
                // products have taken both threads' weights)
                const float top = meet(fmaxf(max3(top4[0], top4[1], top4[2]), top4[3]),
                                       [](float a, float b) { return fmaxf(a, b); }) * p.scale2;
                const bool raise = top > m_ref + (LAZY + T::first_weight);
                const float m_new = top - T::first_weight;
                if (__builtin_expect(j > 0 && __any_sync(0xFFFFFFFFu, raise), 0)) {
                    wait(sh, &sh.pv_done[t][(met - 1) % SB], ((met - 1) / SB) & 1);  // the output is free
                    tc_fence_after();
                    const float f = raise ? ex2(m_ref - m_new) : 1.0f;
                    l *= f;
#pragma unroll 1
                    for (int c = half * (NC * 64 / HALVES); c < (half + 1) * (NC * 64 / HALVES); c += 16) {
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
                    tmem_st16(s_b + half * (C / 2) + 16 * c, w);
                }
                tmem_wait_st();
                tc_fence_before();
                // (an arrival a warp: 128 of them took the barriers' unit longer than the weights)
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_ready[t][buffer]);
                float l0, l1;
                unpack2(add2(part[0], part[1]), l0, l1);
                l += l0 + l1;
            }
            if (nt > 0) {
                wait_long(sh, &sh.pv_done[t][(met - 1) % SB], ((met - 1) / SB) & 1);
                tc_fence_after();
            }
            l = meet(l, [](float a, float b) { return a + b; });
            // (a sum of zero: nothing was seen; one that is NaN stays so)
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const float lse2 = l == 0.0f ? -INFINITY : m_ref + log2f(l);
            const int h = my.head * p.G + r - my_tok * p.G;
            const bool real = r < p.tile_rows && tok < my.u.nq;
            const bool whole = i0 == 0 && my.i1 == my.n;
            const int64_t out_row = my.u.q0 + tok;
            const int slot_out = 2 * blockIdx.x + (i0 > 0 ? 0 : 1);
            if (real && half == 0) {
                if (!whole)
                    p.part_lse[static_cast<int64_t>(slot_out) * (NT * TM) + t * TM + r] = lse2;
                else if (p.lse)
                    p.lse[out_row * p.Hq + h] = lse2 * LN2;
            }
            // A warp's 32 rows x 32 columns go through shared memory, so that four lanes write 64
            // bytes of a row.
            const uint32_t stage = q_s + Z::STAGES + (warp - 4) * Z::STAGE;
            const int64_t mine = reinterpret_cast<int64_t>(p.out + out_row * p.out_tok + h * p.out_head);
#pragma unroll 1
            for (int col = half * (NC * 64 / HALVES); col < (half + 1) * (NC * 64 / HALVES); col += 32) {
                uint32_t o[32];
                tmem_ld32(o_t + col, o);
                tmem_wait_ld();
                // (where no key was met, the columns hold anything)
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = nt > 0 ? __float_as_uint(__uint_as_float(o[i]) * inv) : 0u;
                if (!whole) {
                    if (real)
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *part_at<NC, TM, NT>(p, slot_out, t, col + i, r) =
                                make_float4(__uint_as_float(o[i]), __uint_as_float(o[i + 1]),
                                            __uint_as_float(o[i + 2]), __uint_as_float(o[i + 3]));
                    continue;
                }
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    uint32_t y[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        y[u] = T::narrow2(__uint_as_float(o[8 * v + 2 * u]), __uint_as_float(o[8 * v + 2 * u + 1]));
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                     stage + lane * 64 + ((v ^ ((lane >> 1) & 3)) << 4)),
                                 "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
                                 : "memory");
                }
                __syncwarp();
                const bool in = col + (lane & 3) * 8 < p.D;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int row = k * 8 + lane / 4;
                    uint4 y;
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w)
                                 : "r"(stage + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4))
                                 : "memory");
                    const int64_t to = __shfl_sync(0xFFFFFFFFu, mine, row) + (col + (lane & 3) * 8) * 2;
                    if (__shfl_sync(0xFFFFFFFFu, static_cast<int>(real), row) && in)
                        *reinterpret_cast<uint4 *>(to) = y;
                }
                __syncwarp();
            }
            // The next item's products overwrite this output once its first weights are there,
            // which come after these reads.
            tc_fence_before();
            __syncwarp();  // the whole warp is done with the item
            if (lane == 0) mbar_arrive(&sh.item_free[item % ITEMS]);
        }
    } else if (warp == 0) {
        // ---- producer: a box of a tile a lane.  Tiles are numbered through all items of the CTA,
        // and tile j takes slot j mod RING.
        const int boxes = TN / p.box_rows;
        const uint32_t q_bytes = NC * p.tile_rows * 128;
        uint32_t j = 0, q_uses[2] = {0, 0};
        const auto all = [](bool yes) { return __all_sync(0xFFFFFFFFu, yes) != 0; };
        const auto wait_all = [&](uint64_t *bar, uint32_t parity) {  // one lane asks
            return all(lane != 0 || wait(sh, bar, parity));
        };
        bool ok = true;
        for (uint32_t item = 0; ok && all(there_is(item)); ++item) {
            const Item my = sh.item[item % ITEMS];
            const int n = my.tiles();
            // the page of this lane's box of the item's tile i
            const int32_t *table = p.block_table + static_cast<int64_t>(my.row) * p.max_pages;
            Box box = {};
            const auto look = [&](int i) {
                box.look(p, table, my.u.key_tile(my.i0 + i) * TN + lane * p.box_rows, my.u.len, lane < boxes);
            };
            // a tile's keys or values into their slot, once that is free
            const auto bring = [&](const CUtensorMap *map, uint64_t *full, uint64_t *free, int chunk, int2 at) {
                if (j >= RING && !wait_all(free, (j / RING - 1) & 1)) return false;
                if (lane == 0) mbar_expect_tx(full, NC * CHUNK);
                __syncwarp();
                const uint32_t dst = ring + j % RING * Z::TILE + chunk * CHUNK + lane * p.box_rows * 128;
                if (lane < boxes)
#pragma unroll
                    for (int c = 0; c < NC; ++c)
                        tma_load_4d(dst + c * CHUNK, map, c * 64, at.y, my.head, at.x, full);
                __syncwarp();
                return true;
            };
            if (n > 0) look(0);
            for (int i = 0; ok && i < n; ++i, ++j) {
                const int2 to = box.settle(p);
                if (i + 1 < n) look(i + 1);
                const uint32_t slot = j % RING;
                ok = bring(&maps.k, &sh.k_full[slot], &sh.k_free[slot], 0, to);
                if (ok && i == 0) {  // the queries, behind the first keys, which wait for less
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        if (my.nt[t] > 0) {
                            ok = ok && (q_uses[t] == 0 || wait_all(&sh.q_free[t], (q_uses[t] - 1) & 1));
                            if (!ok) break;
                            ++q_uses[t];
                            if (lane == 0) {
                                mbar_expect_tx(&sh.q_full[t], q_bytes);
                                for (int c = 0; c < NC; ++c)
                                    tma_load_4d(q_s + (t * NC + c) * Q_CHUNK, &maps.q, c * 64, 0,
                                                my.u.q0 + (my.u.m0 + t * p.tile_rows) / p.G, my.head, &sh.q_full[t]);
                            }
                            __syncwarp();
                        }
                }
                ok = ok && bring(&maps.v, &sh.v_full[slot], &sh.v_free[slot], NC, to);
            }
            __syncwarp();  // (all lanes have read the item)
            if (lane == 0) mbar_arrive(&sh.item_free[item % ITEMS]);
        }
        if (__any_sync(0xFFFFFFFFu, sh.abort)) {
            // let the copies in flight land: the last fills of every slot, and the queries' (a fill
            // that was cut off never completes: its wait runs to the limit)
            for (uint32_t i = j > RING ? j - RING : 0; i < j; ++i) {
                wait_out(&sh.k_full[i % RING], (i / RING) & 1);
                wait_out(&sh.v_full[i % RING], (i / RING) & 1);
            }
            for (int t = 0; t < NT; ++t)
                if (q_uses[t] > 0) wait_out(&sh.q_full[t], (q_uses[t] - 1) & 1);
        }
    } else if (warp == 1) {
        if (elect_one()) {
            // ---- MMA issuer: a tile's products, then the next scores of the same rows, in turn
            constexpr uint32_t id_s = idesc_of<T>(TN, false), id_o = idesc_of<T>(NC * 64, true);
            const uint64_t qd = smem_desc_sw128(q_s), kd = smem_desc_sw128(ring);
            const uint64_t vd = smem_desc_rows_k(ring, CHUNK) + NC * (CHUNK >> 4);
            // the numbers of the next key tile, and of the next one that a row tile meets, for the
            // products and for the scores
            uint32_t gv = 0, gk = 0, mv[2] = {0, 0}, mk[2] = {0, 0}, q_uses[2] = {0, 0};
            for (uint32_t item = 0; there_is(item); ++item) {
                const int nt[2] = {sh.item[item % ITEMS].nt[0], sh.item[item % ITEMS].nt[1]}, n = max(nt[0], nt[1]);
                for (int j = -SB; j < n && !sh.abort; ++j) {
                    const uint32_t vs = gv % RING, ks = gk % RING;
                    if (j >= 0 && !wait(sh, &sh.v_full[vs], (gv / RING) & 1)) break;
                    bool keys = false;  // tile j + SB's have been waited for
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        if (j >= 0 && j < nt[t]) {
                            if (!wait(sh, &sh.p_ready[t][mv[t] % SB], (mv[t] / SB) & 1)) break;
                            tc_fence_after();
                            const uint32_t a_d = tmem + t * 128 + mv[t] % SB * TN, d = tmem + O_COL + t * 128;
                            const uint64_t b_d = vd + vs * (Z::TILE >> 4);
#pragma unroll
                            for (int u = 0; u < TN / 16; ++u)
                                mma_ts(d, a_d + 8 * u, b_d + u * (2048 >> 4), id_o, (j | u) != 0);
                            mma_commit(&sh.pv_done[t][mv[t] % SB]);
                            ++mv[t];
                        }
                        if (t == NT - 1 && j >= 0) mma_commit(&sh.v_free[vs]);
                        if (j + SB < nt[t]) {
                            if (!keys && !wait(sh, &sh.k_full[ks], (gk / RING) & 1)) break;
                            keys = true;
                            if (j == -SB && !wait(sh, &sh.q_full[t], q_uses[t]++ & 1)) break;
                            const uint32_t d = tmem + t * 128 + mk[t] % SB * TN;
                            const uint64_t a_d = qd + t * (NC * (Q_CHUNK >> 4)), b_d = kd + ks * (Z::TILE >> 4);
#pragma unroll
                            for (int c = 0; c < NC; ++c)
#pragma unroll
                                for (int u = 0; u < 4; ++u)
                                    mma_bf16(d, a_d + c * (Q_CHUNK >> 4) + 2 * u, b_d + c * (CHUNK >> 4) + 2 * u, id_s,
                                             (c | u) != 0);
                            mma_commit(&sh.s_full[t][mk[t] % SB]);
                            if (j + SB + 1 == nt[t]) mma_commit(&sh.q_free[t]);
                            ++mk[t];
                        }
                    }
                    if (keys) {
                        mma_commit(&sh.k_free[ks]);
                        ++gk;
                    }
                    gv += j >= 0;
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
            it.g0 += it.tiles();
#pragma unroll
            for (int t = 0; t < 2; ++t) it.met[t] += it.nt[t];
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
    const size_t rows = static_cast<size_t>(2 * SMS) * TM * (NC <= 2 ? 2 : 1);
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
    if (!set_up(a, TM / G * G, Z::NT, Z::TN, true, y.plan, y.part, y.lse, p, maps)) return cudaErrorInvalidValue;
    static AttrCache attr;
    cudaError_t e = ensure_attr(k_heads_chunk<T, NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, Z::SMEM, attr);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(SMS);
    cfg.blockDim = dim3(Z::THREADS);
    cfg.dynamicSmemBytes = Z::SMEM;
    cfg.stream = stream;
    cfg.attrs = pdl_attr();  // set up beside the end of whatever the stream runs before
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_heads_chunk<T, NC>, maps, p);
    if (e != cudaSuccess) return e;
    count_launches(1);
    cfg.gridDim = dim3(Z::NT * TM / 32, SMS);
    cfg.blockDim = dim3(JOIN_THREADS);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, k_heads_join<T, NC, TM, Z::NT, false>, p);
    if (e == cudaSuccess) count_launches(1);
    return e;
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
