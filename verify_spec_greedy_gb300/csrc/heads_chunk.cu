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

#include "heads.cuh"

namespace mtpspec {
namespace hch {

using namespace heads;

constexpr int TM = 128;            // rows of a tile in tensor memory
constexpr int TN = 128;            // keys of a tile
constexpr int CHUNK = TN * 128;    // bytes of 128 rows x 64 columns of 16 bits
constexpr int NTHREADS = 640;      // warp 0 TMA, 1 MMA, 2 next work, 3 TMEM; 4-11, 12-19 softmax
constexpr uint32_t TMEM_COLS = 512;
constexpr int S_COL = 0, O_COL = 256;  // tile t: + 128 t

// An item of a CTA: tiles i0 .. i1 - 1 of a unit's list; with the key tiles before it, and the
// items before it in which either row tile had keys to meet, and the key tiles that it met (as
// far as parities go).  head -1: no more.
struct Item {
    Unit<TN> u;
    int row, head, i0, i1, n;   // n: the unit's tiles, at least 1
    uint32_t g0, outputs[2], met[2];
};

struct __align__(16) Shared {
    uint64_t k_full[2], v_full[2], k_free[2], v_free[2];  // by the tile's number mod 2
    uint64_t q_full[2], q_free[2], s_full[2], p_ready[2], o_done[2], v_clean, drained;
    uint64_t item_full[2], item_free[2];
    Item item[2];
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

// What an item's row tiles and its producer go by.
struct Extent {
    int n0, n1, n, tail;
    __device__ __forceinline__ Extent(const Params &p, const Item &it) {
        n0 = max(0, min(it.i1, it.u.tiles(p, it.u.m0, p.tile_rows)) - it.i0);
        n1 = max(0, min(it.i1, it.u.tiles(p, it.u.m0 + p.tile_rows, p.tile_rows)) - it.i0);
        n = max(n0, n1);
        tail = it.u.tail() - it.i0;  // as far as the item meets it
        if (tail >= n) tail = -1;
    }
    __device__ __forceinline__ int tiles(int t) const { return t ? n1 : n0; }
    // the tile of rows that uses every chunk last
    __device__ __forceinline__ int last() const { return n1 >= n0 ? 1 : 0; }
};
template <int NC>
struct Sizes {
    static constexpr int TILE = 2 * NC, RING = 2 * TILE;   // chunks of a tile's keys and values
    static constexpr int EXTRA = static_cast<int>(sizeof(Shared));
    // (more than half of an SM's, so that no two CTAs, which take all its tensor memory, share one)
    static constexpr int SMEM = ((2 * NC + RING) * CHUNK > 120 * 1024 ? (2 * NC + RING) * CHUNK : 120 * 1024) + EXTRA;
    static constexpr int COLS = 64 * NC;
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
    // ---- where this CTA starts, and its first item
    Walk<TN> walk;
    const Cut cut = find_start<TN, NTHREADS>(p, sh.scan, 2, walk);
    const auto next = [&](Item &it) {
        const bool more = walk.next(p, cut, it.u, it.i0, it.i1, it.n);
        it.row = walk.row;
        it.head = more ? walk.head : -1;
        return more;
    };
    if (warp == 2) {
        Item it = {};
        next(it);
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
        const int my_tok = r / p.G, last_tok = p.tile_rows / p.G - 1;  // within the tile
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
                it.u.m0 = my.u.m0;
                it.u.w0 = my.u.w0;
                it.u.ns = my.u.ns;
                it.i0 = i0 = my.i0;
                it.i1 = my.i1;
                const Extent e(p, it);
                nt = e.tiles(t);
                tail = e.last() == t ? e.tail : -1;  // the tile whose values are to be cleared
                sure = it.u.len - it.u.nq + (it.u.m0 + t * p.tile_rows) / p.G + 1;  // the least limit of the tile's rows
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
                if (__builtin_expect(key0 + TN > sure || (width && key0 < sure + last_tok - width), 0)) {
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
            const int tok = (my.u.m0 + t * p.tile_rows) / p.G + my_tok, h = my.head * p.G + r - my_tok * p.G;
            const bool real = r < p.tile_rows && tok < my.u.nq;
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
        const uint32_t q_bytes = NC * p.tile_rows * 128;
        uint32_t j = 0, q_uses[2] = {0, 0};
        const auto all = [](bool yes) { return __all_sync(0xFFFFFFFFu, yes) != 0; };
        for (uint32_t item = 0;; ++item) {
            const Item my = sh.item[item & 1];
            const Extent x(p, my);
            // the page of this lane's box of the item's tile i
            const int32_t *table = p.block_table + static_cast<int64_t>(my.row) * p.max_pages;
            int2 box = {};
            const auto look = [&](int i) {
                box = find_box(p, table, my.u.key_tile(my.i0 + i) * TN + lane * p.box_rows, my.u.len, lane < boxes);
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
                                        my.u.q0 + (my.u.m0 + t * p.tile_rows) / p.G, my.head, &sh.q_full[t]);
                    }
                    __syncwarp();
                }
            for (int i = 0; ok && i < x.n; ++i, ++j) {
                const int2 to = box;
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
                        tma_load_4d(dst + c * CHUNK, &maps.k, c * 64, my.head, to.y, to.x, &sh.k_full[half]);
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
                        tma_load_4d(dst + (NC + c) * CHUNK, &maps.v, c * 64, my.head, to.y, to.x,
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
    if (warp == 2) walk.close(p);
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
Layout layout(int32_t D) {
    const auto align256 = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
    Layout y;
    y.plan = 0;
    y.part = align256(SMS * sizeof(Plan));
    y.lse = y.part + static_cast<size_t>(2 * SMS) * 2 * TM * ((D + 63) / 64 * 64) * 4;
    y.total = y.lse + align256(static_cast<size_t>(2 * SMS) * 2 * TM * 4);
    return y;
}

template <typename T, int NC>
cudaError_t launch(const Maps &maps, const Params &p, cudaStream_t stream) {
    constexpr int smem = Sizes<NC>::SMEM;
    static AttrCache attr;
    cudaError_t e = ensure_attr(k_heads_chunk<T, NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem, attr);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(SMS);
    cfg.blockDim = dim3(NTHREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = pdl_attr();  // set up beside the end of whatever the stream runs before
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_heads_chunk<T, NC>, maps, p);
    if (e != cudaSuccess) return e;
    count_launches(1);
    cfg.gridDim = dim3(2 * TM / JOIN_WARPS, SMS);
    cfg.blockDim = dim3(JOIN_THREADS);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, k_heads_join<T, NC, TM, 2>, p);
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
    heads::Params p;
    heads::Maps maps;
    const int G = a.Hq / a.Hkv, tok = hch::TM / G;
    const hch::Layout y = hch::layout(a.D);
    if (!heads::set_up(a, tok * G, 2, hch::TN, y.plan, y.part, y.lse, p, maps)) return cudaErrorInvalidValue;
    return dtype == MTPSPEC_BF16 ? hch::pick<Bf16>(maps, p, stream) : hch::pick<F16>(maps, p, stream);
}

}  // namespace mtpspec
