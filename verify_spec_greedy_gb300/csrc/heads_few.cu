// Attention with grouped heads over the paged cache, for batches of few tokens a row (on average: a long
// row among them is cut into units of 32 rows like any other) and heads of up to 64 elements: draft steps
// and verifications.  What bounds them is the cache's bytes and, at 32 KB a tile of keys and values, the way
// from one tile to the next.
//
// One pass over the keys with the running maximum m and sum l of a softmax, as in heads_chunk.cu.
// A unit's rows, the (token, head) rows of a key head, are 32, whose accumulators are folded into all
// 128 lanes of tensor memory: four threads share a row, so that with few rows every thread of the
// four softmax warps has work, 32 keys of a tile each.
//
// Keys and values stream through a ring of chunks (128 tokens x 64 columns), released one by one.
// The scores of a tile are computed ahead of the weights of the tile before, across units as well.
// Two CTAs share an SM: while one is in a softmax, the other's copies and products go on.
//
// What bounds it (HBM copy 6.8 TB/s measured; in a graph): 64 rows of a token, 64 / 8 heads of 64, pages of
// 16, a window of 1024 and four first tokens, fp16, 136 MB: 37 us, 3.6 TB/s (in the other kernel 49); 160
// MB are read.  512 units of ten tiles on 304 CTAs: starts, ends and joins of units cut once or twice each.
// (Two producers, two buffers of weights: the same.)
#include <algorithm>

#include "heads.cuh"

namespace mtpspec {
namespace hfw {

using namespace heads;

constexpr int ROWS = 32, TN = 128;  // rows of a unit, keys of a tile
constexpr int NQ = 128 / ROWS;       // threads of a row
constexpr int C = TN / NQ;           // keys of a tile that a thread has
constexpr int W = 64 / NQ;           // and columns of the output
constexpr int CHUNK = TN * 128;      // bytes of a tile's keys, or values
constexpr int Q_BYTES = ROWS * 128;
constexpr int P_BYTES = TN / 64 * ROWS * 128;
constexpr int CTAS = 2;              // of an SM
constexpr int S_COL = 0, O_COL = 2 * C;
constexpr uint32_t TMEM_COLS = 128;
static_assert(O_COL + W <= static_cast<int>(TMEM_COLS), "tensor memory");
constexpr int NTHREADS = 224;  // warp 0 TMA, 1 MMA and TMEM, 2-5 softmax, 6 items and queries
constexpr int SOFTMAX0 = 64, SOFTMAX = 128;  // the first softmax thread, and how many
constexpr int SLOTS = 5;             // chunks of the ring

// Tiles i0 .. i1 - 1 of a unit's n (at least 1).  head -1: no more.
struct Item {
    Unit<TN> u;
    int row, head, i0, i1, n, tiles;
};

struct __align__(16) Shared {
    uint64_t full[SLOTS], empty[SLOTS];
    uint64_t s_full[2], p_ready, pv_done, q_full[2], item_full[2], item_free[2], drained;
    Item item[2];
    Scan scan;
    int2 box[2][16];  // boxes of a tile, in turn
    uint32_t tmem;
    volatile int abort;
    float other[2][NQ][ROWS];  // what the threads of a row tell each other
};

constexpr int EXTRA = static_cast<int>(sizeof(Shared));
constexpr int SMEM = 2 * Q_BYTES + P_BYTES + SLOTS * CHUNK + EXTRA;
static_assert(SMEM <= 113 * 1024 && SMEM > 75 * 1024, "two CTAs an SM, and no more: they take a quarter of its tensor memory");

// The slot n chunks on, and its phase.
__device__ __forceinline__ void step(int &s, uint32_t &ph, int n) {
    s += n;
    if (s >= SLOTS) {
        s -= SLOTS;
        ph ^= 1;
    }
}

template <typename T>
__global__ void __launch_bounds__(NTHREADS, CTAS)
k_heads_few(const __grid_constant__ Maps maps, const Params p) {
    extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle's period
    const uint32_t q_s = smem_addr(smem), p_s = q_s + 2 * Q_BYTES, ring = p_s + P_BYTES;
    Shared &sh = *reinterpret_cast<Shared *>(smem + SMEM - EXTRA);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == 0) {
        if (lane < SLOTS) {
            mbar_init(&sh.full[lane], 1);
            mbar_init(&sh.empty[lane], 1);
        } else if (lane == 16) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(&sh.s_full[i], 1);
                mbar_init(&sh.q_full[i], 1);
                mbar_init(&sh.item_full[i], 1);
                mbar_init(&sh.item_free[i], 6);  // the producer, the issuer, four softmax warps
            }
            mbar_init(&sh.p_ready, 4);
            mbar_init(&sh.pv_done, 1);
            mbar_init(&sh.drained, 1);
            sh.abort = 0;
        } else if (lane == 17) {
            prefetch_map(&maps.k);
            prefetch_map(&maps.v);
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
    Walk<TN> walk;
    const Cut cut = find_start<TN, NTHREADS>(p, sh.scan, 6, walk);
    const auto next = [&](Item &it) {
        const bool more = walk.next(p, cut, it.u, it.i0, it.i1, it.n);
        it.row = walk.row;
        it.head = more ? walk.head : -1;
        it.tiles = more ? max(0, min(it.i1, it.u.tiles(p)) - it.i0) : 0;
        return more;
    };
    if (warp == 6) {
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
    } else if (warp == 0) {
        // ---- producer: a lane finds a box of a tile, and one thread issues all copies
        const int boxes = TN / p.box_rows;
        const auto all = [](bool yes) { return __all_sync(0xFFFFFFFFu, yes) != 0; };
        int s = 0, filled = 0;
        uint32_t ph = 1;  // phase of the slot's release
        bool ok = true;
        for (uint32_t item = 0;; ++item) {
            const Item my = sh.item[item & 1];
            const int32_t *table = p.block_table + static_cast<int64_t>(my.row) * p.max_pages;
            const int window = my.u.window(p);
            Box box = {};
            const auto look = [&](int i) {
                box.look(p, table, my.u.key_tile(my.i0 + i) * TN + lane * p.box_rows, my.u.len, window, lane < boxes);
            };
            if (my.tiles > 0) look(0);
            for (int i = 0; ok && i < my.tiles; ++i) {
                int2 *at = sh.box[i & 1];
                if (lane < boxes) at[lane] = box.settle(p);
                if (i + 1 < my.tiles) look(i + 1);
                __syncwarp();
                if (elect_one()) {
                    int slot = s;
                    uint32_t phase = ph;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {  // the keys, then the values
                        ok = ok && wait(sh, &sh.empty[slot], phase);
                        if (!ok) break;
                        mbar_expect_tx(&sh.full[slot], CHUNK);
                        uint32_t dst = ring + slot * CHUNK;
#pragma unroll 4
                        for (int k = 0; k < boxes; ++k) {
                            const int2 x = at[k];
                            tma_load_4d(dst, c == 0 ? &maps.k : &maps.v, 0, x.y, my.head, x.x, &sh.full[slot]);
                            dst += p.box_rows * 128;
                        }
                        step(slot, phase, 1);
                    }
                }
                __syncwarp();
                ok = all(ok);
                filled += 2;
                step(s, ph, 2);
            }
            __syncwarp();  // (all lanes have read the item)
            if (lane == 0) mbar_arrive(&sh.item_free[item & 1]);
            if (!ok || !all(next_item(item))) break;
        }
        if (__any_sync(0xFFFFFFFFu, sh.abort)) {
            // let the copies in flight land (the last fill of each barrier)
            for (int k = 0; k < SLOTS; ++k) {
                const int fills = (filled + SLOTS - 1 - k) / SLOTS;
                if (fills > 0) wait_out(&sh.full[k], (fills - 1) & 1);
            }
        }
    } else if (warp == 1) {
        if (elect_one()) {
            // ---- MMA issuer.  Two kinds of work wait for different things: the scores of tile a
            // for its keys, the products of tile b for its weights and values.  Whichever is there
            // is issued, the products first, since they free slots.
            constexpr uint32_t id_s = idesc_of<T>(ROWS, TN, false), id_o = idesc_of<T>(ROWS, 64, true);
            const uint64_t qd = smem_desc_sw128(q_s), pd = smem_desc_sw128(p_s);
            const uint64_t kd = smem_desc_sw128(ring), vd = smem_desc_rows_k(ring, 16);  // (one chunk: no step)
            int sa = 0, sb = 1;            // the next slots of tile a's keys and tile b's values
            uint32_t pa = 0, pb = 0;        // their phases
            uint32_t ga = 0, gb = 0;        // the numbers of tiles a and b
            uint32_t ahead = 0, firsts = 0, idle = 0;  // tiles between; which are their item's first
            const auto products = [&]() {
                if (ahead == 0 || !mbar_poll(&sh.p_ready, gb & 1) || !mbar_poll(&sh.full[sb], pb)) {
                    if (++idle > POLL_LIMIT) sh.abort = 1;
                    return;
                }
                tc_fence_after();
                const uint64_t v = vd + sb * (CHUNK >> 4);
#pragma unroll
                for (int u = 0; u < TN / 16; ++u)
                    mma_ws(tmem + O_COL, pd + (u >> 2) * (Q_BYTES >> 4) + 2 * (u & 3), v + u * (2048 >> 4), id_o,
                           !(firsts & 1) || u > 0);
                mma_commit(&sh.empty[sb]);
                mma_commit(&sh.pv_done);
                step(sb, pb, 2);
                ++gb;
                --ahead;
                firsts >>= 1;
                idle = 0;
            };
            // waits for a fill, with products between the polls
            const auto filled = [&](uint64_t *bar, uint32_t phase) {
                do {
                    products();
                } while (!mbar_poll(bar, phase) && !sh.abort);
                idle = 0;
                tc_fence_after();
                return !sh.abort;
            };
            for (uint32_t item = 0;; ++item) {
                const int tiles = sh.item[item & 1].tiles;
                mbar_arrive(&sh.item_free[item & 1]);
                const uint64_t q = qd + (item & 1) * (Q_BYTES >> 4);
                if (!filled(&sh.q_full[item & 1], (item >> 1) & 1)) break;
                for (int i = 0; i < tiles && !sh.abort; ++i) {
                    while (ahead > 1 && !sh.abort) products();  // the scores' buffer is free
                    const uint32_t d = tmem + S_COL + (ga & 1) * C;
                    if (!filled(&sh.full[sa], pa)) break;
#pragma unroll
                    for (int u = 0; u < 4; ++u) mma_ws(d, q + 2 * u, kd + sa * (CHUNK >> 4) + 2 * u, id_s, u != 0);
                    mma_commit(&sh.empty[sa]);
                    mma_commit(&sh.s_full[ga & 1]);
                    step(sa, pa, 2);
                    firsts |= static_cast<uint32_t>(i == 0) << ahead;
                    ++ga;
                    ++ahead;
                }
                // (the next item is known one ahead; while it is not, products go on)
                const uint32_t nxt = item + 1;
                uint64_t *bar = &sh.item_full[nxt & 1];
                while (!sh.abort && !mbar_poll(bar, ((nxt - 1) >> 1) & 1)) products();
                idle = 0;
                if (sh.abort || sh.item[nxt & 1].head < 0) break;
            }
            while (ahead > 0 && !sh.abort) products();
            mma_commit(&sh.drained);
            wait_out(&sh.drained, 0);
        }
    } else if (warp == 6) {
        // ---- the items, each published when the one two before it is left behind, and their queries
        Item it = sh.item[0];
        for (uint32_t item = 0;; ++item) {
            const uint32_t to = q_s + (item & 1) * Q_BYTES;
            const int rows = it.u.nq * p.G - it.u.m0;
#pragma unroll 8
            for (int v = lane; v < ROWS * 8; v += 32) {
                const int r = v / 8, cv = v % 8, m = it.u.m0 + r, tok = m / p.G;
                const bool real = r < rows && cv * 8 < p.D;
                const uint16_t *src = p.q + (it.u.q0 + tok) * p.q_tok + (it.head * p.G + m - tok * p.G) * p.q_head + cv * 8;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 to + r * 128 + ((cv ^ (r & 7)) << 4)),
                             "l"(real ? src : p.q), "r"(real ? 16 : 0)
                             : "memory");
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.q_full[item & 1]);
            const bool more = next(it);
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
    } else {
        // ---- softmax: NQ threads a row, C of a tile's keys each
        const int wq = warp & 3, tid = threadIdx.x - SOFTMAX0;
        const int r = (wq * 32 + lane) % ROWS, part = (wq * 32 + lane) / ROWS;
        const uint32_t trow = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        int slot = 0;
        // the threads of a row meet, and each sees the others' values
        const auto meet = [&](float v, auto join) {
            sh.other[slot][part][r] = v;
            asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
            for (int k = 1; k < NQ; ++k) v = join(v, sh.other[slot][(part + k) % NQ][r]);
            slot ^= 1;
            return v;
        };
        uint32_t g = 0;
        for (uint32_t item = 0;; ++item) {
            const volatile Item &my = sh.item[item & 1];
            const int tiles = my.tiles, i0 = my.i0, ns = my.u.ns, skip = my.u.w0 - ns, len = my.u.len;
            const int m0 = my.u.m0, base = len - my.u.nq, rows = my.u.nq * p.G - m0;
            const int tail = (len % TN != 0 ? ns + len / TN - my.u.w0 : -1) - i0;
            const int sure = base + m0 / p.G + 1;             // one past the last key of the first row,
            const int limit = base + (m0 + r) / p.G + 1;      // of this one,
            const int most = base + (m0 + min(ROWS, rows) - 1) / p.G + 1;  // and of the last
            const int width = p.window > 0 && p.window < len ? p.window : 0;
            float m_ref = -INFINITY, l = 0.0f;
            for (int j = 0; j < tiles; ++j, ++g) {
                wait_long(sh, &sh.s_full[g & 1], (g >> 1) & 1);
                tc_fence_after();
                uint32_t x[C];
                tmem_ld32(trow + S_COL + (g & 1) * C, x);
                tmem_wait_ld();
                const int key0 = (i0 + j < ns ? i0 + j : i0 + j + skip) * TN;
                if (__builtin_expect(key0 + TN > sure || (width && key0 < most - width), 0)) {
                    // more than every row sees
                    const int seen = limit - key0 - part * C;
                    const int low = width ? seen - width : -1, first = p.sinks - key0 - part * C;
#pragma unroll
                    for (int i = 0; i < C; ++i)
                        if (i >= seen || (i < low && i >= first)) x[i] = 0xFF800000u;
                }
                float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < C; i += 2)
                    top4[(i >> 1) & 3] = max3(top4[(i >> 1) & 3], __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
                const float top = meet(fmaxf(max3(top4[0], top4[1], top4[2]), top4[3]),
                                       [](float a, float b) { return fmaxf(a, b); }) * p.scale2;
                const bool raise = top > m_ref + (LAZY + T::first_weight);
                const float m_old = m_ref;
                if (raise) m_ref = top - T::first_weight;
                const float m_use = m_ref == -INFINITY ? 0.0f : m_ref;
                const uint64_t scale_2 = pack2(p.scale2, p.scale2), minus_m = pack2(-m_use, -m_use);
                uint64_t sums[2] = {0, 0};  // two pairs of sums
                uint4 weights[C / 8];
#pragma unroll
                for (int v = 0; v < C / 8; ++v) {
                    float e[8];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        float e0, e1;
                        unpack2(fma2(pack2(__uint_as_float(x[8 * v + 2 * u]), __uint_as_float(x[8 * v + 2 * u + 1])),
                                     scale_2, minus_m), e0, e1);
                        e[2 * u] = ex2(e0);
                        e[2 * u + 1] = ex2(e1);
                        sums[u & 1] = add2(sums[u & 1], pack2(e[2 * u], e[2 * u + 1]));
                    }
                    weights[v] = float_to_half8<T>(e);
                }
                // the products of the tile before are done: the weights' buffer and the output are
                // free to change
                if (g > 0) wait(sh, &sh.pv_done, (g - 1) & 1);
                if (__builtin_expect(j > 0 && __any_sync(0xFFFFFFFFu, raise), 0)) {
                    tc_fence_after();
                    const float f = raise ? ex2(m_old - m_ref) : 1.0f;
                    l *= f;
                    uint32_t o[W];
                    tmem_ld16(trow + O_COL, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < W; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                    tmem_st16(trow + O_COL, o);
                    tmem_wait_st();
                }
                float l0, l1;
                unpack2(add2(sums[0], sums[1]), l0, l1);
                l += l0 + l1;
#pragma unroll
                for (int v = 0; v < C / 8; ++v) {
                    const int at = part * (C / 8) + v;  // 16 bytes of the row's 2 TN
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                     p_s + (at >> 3) * Q_BYTES + r * 128 + (((at & 7) ^ (r & 7)) << 4)),
                                 "r"(weights[v].x), "r"(weights[v].y), "r"(weights[v].z), "r"(weights[v].w)
                                 : "memory");
                }
                if (__builtin_expect(j == tail, 0)) {
                    // value rows behind the row's last key: whatever lies there must not meet the
                    // zero weights
                    const int z0 = len % TN;
                    const uint32_t n = 2 * g + 1, at = n % SLOTS;
                    wait(sh, &sh.full[at], (n / SLOTS) & 1);
                    for (int i = tid; i < (TN - z0) * 8; i += 128)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                         ring + at * CHUNK + z0 * 128 + i * 16),
                                     "r"(0)
                                     : "memory");
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_ready);
            }
            // ---- epilogue
            l = meet(l, [](float a, float b) { return a + b; });
            if (tiles > 0) {
                wait(sh, &sh.pv_done, (g - 1) & 1);
                tc_fence_after();
            }
            // (a sum of zero: nothing was seen; one that is NaN stays so)
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const float lse2 = l == 0.0f ? -INFINITY : m_ref + log2f(l);
            const bool real = r < rows, whole = i0 == 0 && my.i1 == my.n;
            const int tok = (m0 + r) / p.G, h = my.head * p.G + m0 + r - tok * p.G;
            const int64_t out_row = my.u.q0 + tok;
            const int slot_out = 2 * blockIdx.x + (i0 > 0 ? 0 : 1);
            if (real && part == 0) {
                if (!whole)
                    p.part_lse[static_cast<int64_t>(slot_out) * ROWS + r] = lse2;
                else if (p.lse)
                    p.lse[out_row * p.Hq + h] = lse2 * LN2;
            }
            uint16_t *dst = p.out + out_row * p.out_tok + h * p.out_head + part * W;
            // 32 bytes a store, a whole sector, where the rows allow it
            const bool sectors = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;
            uint32_t o[W] = {};
            if (tiles > 0) {
                tmem_ld16(trow + O_COL, o);
                tmem_wait_ld();
            }
            if (real) {
                float f[W];
#pragma unroll
                for (int i = 0; i < W; ++i) f[i] = tiles > 0 ? __uint_as_float(o[i]) * inv : 0.0f;
                if (!whole) {
#pragma unroll
                    for (int k = 0; k < W; k += 4)
                        *part_at<1, ROWS>(p, slot_out, part * W + k, r) =
                            make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
                } else if (part * W < p.D) {
                    uint32_t y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = T::narrow2(f[2 * i], f[2 * i + 1]);
                    if (sectors) {
                        st_global_32B(dst, y);
                    } else {
                        *reinterpret_cast<uint4 *>(dst) = make_uint4(y[0], y[1], y[2], y[3]);
                        *reinterpret_cast<uint4 *>(dst + 8) = make_uint4(y[4], y[5], y[6], y[7]);
                    }
                }
            }
            // The next item's products overwrite this output once its first weights are there, which
            // come after these reads.
            tc_fence_before();
            __syncwarp();  // the whole warp is done with the item
            if (lane == 0) mbar_arrive(&sh.item_free[item & 1]);
            if (!all_say<SOFTMAX>(next_item(item), 1)) break;
        }
    }
    if (warp == 6) walk.close(p);
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
        pdl_launch_dependents();
        if (sh.abort && p.status) atomicOr(p.status, MTPSPEC_STATUS_TIMEOUT);
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(TMEM_COLS)
                     : "memory");
    }
}

struct Layout {
    size_t plan, part, lse, total;
};
Layout layout() {
    const auto align256 = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
    constexpr size_t slots = static_cast<size_t>(2) * CTAS * SMS;
    Layout y;
    y.plan = 0;
    y.part = align256(slots * sizeof(Plan));
    y.lse = y.part + slots * ROWS * 64 * 4;
    y.total = y.lse + align256(slots * ROWS * 4);
    return y;
}

template <typename T>
cudaError_t launch(const HeadsAttnArgs &a, cudaStream_t stream) {
    const Layout y = layout();
    Params p;
    Maps maps;
    if (!set_up(a, ROWS, TN, false, y.plan, y.part, y.lse, p, maps)) return cudaErrorInvalidValue;
    static AttrCache attr;
    cudaError_t e = ensure_attr(k_heads_few<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM, attr);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CTAS * SMS);
    cfg.blockDim = dim3(NTHREADS);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = stream;
    cfg.attrs = pdl_attr();  // set up beside the end of whatever the stream runs before
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_heads_few<T>, maps, p);
    if (e != cudaSuccess) return e;
    count_launches(1);
    return launch_join<T, 1, ROWS>(cfg, p, stream);
}

}  // namespace hfw

size_t heads_few_workspace_bytes() { return hfw::layout().total; }

cudaError_t run_heads_few(const HeadsAttnArgs &a, int dtype, cudaStream_t stream) {
    return dtype == MTPSPEC_BF16 ? hfw::launch<Bf16>(a, stream) : hfw::launch<F16>(a, stream);
}

}  // namespace mtpspec
