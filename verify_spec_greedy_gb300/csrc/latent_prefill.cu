// Attention over whole prompts in the expanded form: every head has its own N key values and
// V values a token, and the heads share the R rotated key values of a token.
//
// One pass over the keys with the running maximum m and sum l of a softmax: for a tile of keys
//     S = Q K^T,  p = 2^(s - m),  l += sum p,  O += p V,  and O, l scaled by 2^(m - m') when m
// changes (s, m in powers of two, scale * log2 e folded in; m follows a row's maximum only when
// that has grown by more than 2^8).  Weights are rounded to 16 bits for the second product; l
// sums the unrounded ones in fp32.  (In fp16 m lies 2^7 below that maximum, so that fewer weights
// are subnormal: half_types.cuh.)  Keys that no query of a tile sees are never read.
//
// A pair of query tiles, 256 queries of one head, is a CTA's unit of work: while the tensor
// cores work on one tile's products, the other tile's softmax runs, eight warps a tile, two
// threads a row.  Tensor memory holds both tiles' scores (128 columns each, whose first half
// becomes the weights, the left operand of the second product) and outputs: all of its 512
// columns.  Keys and values stream through a ring of 16 KB chunks (128 tokens x 64 columns) in
// the order in which they are used.  The shared rotated part is read from its own array, so no
// key is ever put together in memory.  The grid has a CTA a pair, and one that has nothing left
// to load takes over a pair whose CTA has not started.
//
// What bounds it (bf16, N = V = 128, R = 64; products 1938 TFLOP/s measured): 8192 tokens x 32
// heads, 687 GFLOP: 477-490 us when called on and on, at the 1815 MHz that the power limit leaves
// (1390 W of 1400), 1.42 PFLOP/s, 0.73; 444 us in the first milliseconds after a pause, at some
// 1900-2070 MHz, 0.80.  Counters: tensor pipe 66 %, shared memory of the products 52 %,
// exponentials 27 %, DRAM 18 %.  A round of both tiles takes some 3,500 cycles
// for 2,560 of products: the chain scores - softmax - products of a tile is longer than the
// other tile's products, and a third tile has no tensor memory.  Splitting the chain (first
// half of the weights handed over early) cost more in barriers than it gave: 439 -> 476 us.
// 8 prompts of 77-1500 tokens x 32 heads, 61 GFLOP: 85 us, 0.71 PFLOP/s: the last softmax and
// the output of a pair are not covered by anything (tensor pipe 34 %), and tiles on the diagonal
// and at the ends are computed whole, 1.27 times the visible products.  Two chunks of 900 and
// 1000 queries x 16 heads behind 7001 keys: 129-135 us, 1.11-1.14 PFLOP/s: 128 pairs, 24 of the 152
// multiprocessors have none.  300 tokens x 16 heads: 12 us, the way from launch to output.
//
// Registers: 640 threads leave 96 a thread, and each instance spills 48 or 52 bytes a thread.
#include <algorithm>

#include "half_types.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace mtpspec {
namespace lpf {

using namespace tg;

constexpr int TM = 128;            // queries of a tile
constexpr int TN = 128;            // keys of a tile
constexpr int CHUNK = TN * 128;    // bytes of 128 rows x 64 columns of 16 bits
constexpr int NTHREADS = 640;      // warp 0 TMA, 1 MMA, 2 next work, 3 TMEM; 4-11, 12-19 softmax
constexpr int SMEM_MAX = 232448;   // 227 KB a CTA
constexpr float LAZY = 8.0f;       // the running maximum may lag by a factor of 2^8
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr uint32_t TMEM_COLS = 512;
constexpr int S_COL = 0, O_COL = 256;  // tile t: + 128 t
constexpr uint32_t POLL_LIMIT = 1u << 25;  // polls of some 20 ns: ~1 s

struct Params {
    const int32_t *cu_q, *cu_k;
    int B, Tq, Tk, Hq, N, R, V;
    int ranks;      // query tiles (pairs) a head has at most
    float scale2;   // scale * log2(e), above 0
    uint16_t *out;
    int64_t out_tok, out_head;
    float *lse;
    int32_t *status;
};

// A pair of query tiles of one head: its sequence, and its place there; pair -1: none.
struct Work {
    int q0, nq, k0, nk, pair, head;
};
// The same as the CTA's roles get it: with the key tiles before it, the ring's slot that it
// starts in, and the pairs before it in which either tile of queries had keys to meet, and
// the key tiles that it met (as far as parities go).
struct Item {
    Work w;
    uint32_t g0;
    int slot0;
    uint32_t outputs[2], met[2];
};

struct __align__(16) Shared {
    uint4 taken;  // the answer to a request for another CTA's work
    // a tile's keys (rotated part included) and its values, by the tile's number mod 2
    uint64_t k_full[2], v_full[2], k_free[2], v_free[2];
    uint64_t q_full[2], q_free[2], s_full[2], p_ready[2], o_done[2], v_clean, drained;
    uint64_t near_end, answer, item_full[2], item_free[2];
    Item item[2];
    uint32_t tmem;
    volatile int abort;
    float other[2][2][TM];  // what the two threads of a row tell each other, by tile and half
};
constexpr int SMEM_EXTRA = static_cast<int>(sizeof(Shared));

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

// And for one on others whose own waits are bounded, which may take as long as a whole pair, or as
// the requests for all CTAs that have no work.
__device__ __forceinline__ bool wait_far(Shared &sh, uint64_t *bar, uint32_t parity,
                                        uint32_t limit = 16 * WAIT_LIMIT) {
    for (uint32_t it = 0; it < limit; ++it) {
        if (mbar_test(bar, parity)) return true;
        if (sh.abort) return false;
    }
    sh.abort = 1;
    return false;
}

// The bounded wait of a CTA that leaves, whatever the abort flag says.
__device__ __forceinline__ void wait_out(uint64_t *bar, uint32_t parity) {
    for (uint32_t it = 0; it < WAIT_LIMIT; ++it)
        if (mbar_test(bar, parity)) return;
}

// Bound i of `cu` as it is taken: in [0, n], and not below the ones before it (as taken, `before`,
// at least 0), so that sequences never overlap and have no more pairs than the grid has CTAs.
__device__ __forceinline__ int bound(const int32_t *cu, int i, int n, int before) {
    return max(min(cu[i], n), before);
}

__device__ __forceinline__ int pairs_of(int queries) { return (queries + 2 * TM - 1) / (2 * TM); }

// A lane's run of sequences b0 .. b1 - 1: the largest bounds before its first (0 when all bounds
// are in range and in order, as they should be), the pairs before it and its own.
struct Run {
    int b0, b1, q_before, k_before, at, sum;
};

// The pair of number `rank`, for a warp whose lanes hold the runs.  Up to 32 sequences (one a
// lane), pairs go by their place in their sequence, the furthest first; beyond, sequence by
// sequence.
__device__ __forceinline__ Work find_work(const Params &p, const Run &run, int rank, int head) {
    Work w = {0, 0, 0, 0, -1, head};
    const int sum = run.sum;
    int at = run.at;
    bool mine = at <= rank && rank < at + sum;
    int pair = at + sum - 1 - rank;
    if (p.B > 1 && p.B <= 32) {
        mine = false;
        pair = sum;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) pair = max(pair, __shfl_xor_sync(0xFFFFFFFFu, pair, o));
        while (--pair >= 0) {
            const unsigned has = __ballot_sync(0xFFFFFFFFu, sum > pair);
            const int n = __popc(has);
            if (rank < n) {
                const unsigned below = has & ((1u << (threadIdx.x & 31)) - 1);
                mine = sum > pair && __popc(below) == rank;
                break;
            }
            rank -= n;
        }
    }
    if (mine) {
        int q0 = bound(p.cu_q, run.b0, p.Tq, run.q_before), k0 = bound(p.cu_k, run.b0, p.Tk, run.k_before);
        for (int b = run.b0; b < run.b1; ++b) {
            const int q1 = bound(p.cu_q, b + 1, p.Tq, q0), k1 = bound(p.cu_k, b + 1, p.Tk, k0);
            const int n = pairs_of(q1 - q0);
            if (p.B <= 32 || rank < at + n) {
                w = {q0, q1 - q0, k0, k1 - k0, p.B <= 32 ? pair : n - 1 - (rank - at), head};
                break;
            }
            at += n;
            q0 = q1;
            k0 = k1;
        }
    }
    const unsigned who = __ballot_sync(0xFFFFFFFFu, mine);
    const int src = who ? __ffs(who) - 1 : 0;
    w.q0 = __shfl_sync(0xFFFFFFFFu, w.q0, src);
    w.nq = __shfl_sync(0xFFFFFFFFu, w.nq, src);
    w.k0 = __shfl_sync(0xFFFFFFFFu, w.k0, src);
    w.nk = __shfl_sync(0xFFFFFFFFu, w.nk, src);
    w.pair = __shfl_sync(0xFFFFFFFFu, w.pair, src);
    return w;
}

// The request for the work of a CTA that has not started (which then never does), and what it
// gave: that CTA's number, or -1 when there is none left.  After a -1 no more may be asked.
__device__ __forceinline__ void ask_for_work(uint4 *dst, uint64_t *bar) {
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
            smem_addr(dst)),
        "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ int work_given(const uint4 *src) {
    int cta;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
        "ld.shared.b128 h, [%1];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "mov.b32 %0, -1;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, h;\n\t}"
        : "=r"(cta)
        : "r"(smem_addr(src))
        : "memory");
    return cta;
}

// How far a pair of query tiles reaches: its first query's place in the sequence, and the key
// tiles that either tile meets (a tile's last query sees the most).
struct Extent {
    int row0, n0, n1, n, nk;
    __device__ __forceinline__ Extent(const Work &w) : row0(w.pair * 2 * TM), nk(w.nk) {
        n0 = met(w, 0);
        n1 = met(w, 1);
        n = max(n0, n1);
    }
    __device__ __forceinline__ int met(const Work &w, int t) const {
        const int first = row0 + t * TM, end = min(first + TM, w.nq);
        const int seen = end + w.nk - w.nq;
        return first >= w.nq || seen <= 0 ? 0 : (seen + TN - 1) / TN;
    }
    __device__ __forceinline__ int tiles(int t) const { return t ? n1 : n0; }
    // the tile of queries that uses every chunk last
    __device__ __forceinline__ int last() const { return n1 >= n0 ? 1 : 0; }
    // the tile that the sequence's keys end in, if the pair meets it and it is not a whole one
    __device__ __forceinline__ int tail() const { return nk % TN != 0 && nk / TN < n ? nk / TN : -1; }
};

// What follows from the chunks of a key tile and of a value tile.
template <int KC, int VC>
struct Sizes {
    static constexpr int LEFT = (SMEM_MAX - SMEM_EXTRA) / CHUNK - 2 * KC;
    static constexpr int TILE = KC + VC, SLOTS = LEFT < 2 * TILE ? LEFT : 2 * TILE;
    static constexpr int SMEM = (2 * KC + SLOTS) * CHUNK + SMEM_EXTRA;
    static_assert(SLOTS > TILE, "a tile and the start of the next");
    // the slot `n` behind slot s of the ring
    static __device__ __forceinline__ int behind(int s, int n) {
        return s + n >= SLOTS ? s + n - SLOTS : s + n;
    }
};

// KC, VC: the 64-column chunks of a key tile (N / 64 + 1 with the rotated one) and of a value
// tile (V / 64).
template <typename T, int KC, int VC>
__global__ void __launch_bounds__(NTHREADS, 1)
k_latent_prefill(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mkv,
                 const __grid_constant__ CUtensorMap mrot, const Params p) {
    extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle's period
    using Z = Sizes<KC, VC>;
    const uint32_t q_s = smem_addr(smem), ring = q_s + 2 * KC * CHUNK;
    Shared &sh = *reinterpret_cast<Shared *>(smem + Z::SMEM - SMEM_EXTRA);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // ---- warp 2 finds work, from a scan of the sequences' pairs with a run of sequences a lane.
    // Work goes by rank: heads side by side, the longest pairs of all of them first, so that
    // what is left at the end is short, and CTAs that share a head's keys walk them at the
    // same time.
    Run run = {};
    int pairs = 0;
    const auto work_of = [&](int cta) {
        const int rank = cta / p.Hq;
        return rank < pairs ? find_work(p, run, rank, cta % p.Hq) : Work{0, 0, 0, 0, -1, 0};
    };
    if (warp == 2) {
        const int per = (p.B + 31) / 32;
        run.b0 = min(p.B, lane * per);
        run.b1 = min(p.B, run.b0 + per);
        int q0 = p.cu_q[run.b0], k0 = p.cu_k[run.b0];
        bool good = q0 >= 0 && k0 >= 0 && q0 <= p.Tq && k0 <= p.Tk;
        for (int b = run.b0; b < run.b1; ++b) {
            const int q1 = p.cu_q[b + 1], k1 = p.cu_k[b + 1];
            good &= q1 >= q0 && k1 >= k0 && q1 <= p.Tq && k1 <= p.Tk;
            if (good) run.sum += pairs_of(q1 - q0);
            q0 = q1;
            k0 = k1;
        }
        if (!__all_sync(0xFFFFFFFFu, good)) {  // each bound counts as the largest up to it
            if (blockIdx.x == 0 && lane == 0 && p.status) atomicOr(p.status, MTPSPEC_STATUS_BAD_PARAM);
            int q = 0, k = 0;
            for (int b = run.b0; b < run.b1; ++b) {
                q = bound(p.cu_q, b, p.Tq, q);
                k = bound(p.cu_k, b, p.Tk, k);
            }
            for (int o = 1; o < 32; o <<= 1) {  // (lanes without one to their left get their own)
                q = max(q, __shfl_up_sync(0xFFFFFFFFu, q, o));
                k = max(k, __shfl_up_sync(0xFFFFFFFFu, k, o));
            }
            q = __shfl_up_sync(0xFFFFFFFFu, q, 1);
            k = __shfl_up_sync(0xFFFFFFFFu, k, 1);
            run.q_before = lane > 0 ? q : 0;
            run.k_before = lane > 0 ? k : 0;
            run.sum = 0;
            q = bound(p.cu_q, run.b0, p.Tq, run.q_before);
            for (int b = run.b0; b < run.b1; ++b) {
                const int q1 = bound(p.cu_q, b + 1, p.Tq, q);
                run.sum += pairs_of(q1 - q);
                q = q1;
            }
        }
        run.at = run.sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, run.at, o);
            if (lane >= o) run.at += v;
        }
        pairs = __shfl_sync(0xFFFFFFFFu, run.at, 31);
        run.at -= run.sum;
        const Work w = work_of(blockIdx.x);
        if (lane == 0) sh.item[0] = Item{w, 0, 0, {0, 0}, {0, 0}};
    }
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
        }
        mbar_init(&sh.v_clean, 256);
        mbar_init(&sh.drained, 1);
        mbar_init(&sh.near_end, 1);
        mbar_init(&sh.answer, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.item_full[i], 1);
            mbar_init(&sh.item_free[i], 18);  // the producer, the issuer, sixteen softmax warps
        }
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&mq);
        prefetch_map(&mkv);
        prefetch_map(&mrot);
    }
    if (warp == 3) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(&sh.tmem)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    // Every role goes through the CTA's items: is there one after number `item`, and no abort?
    const auto next_item = [&](uint32_t item) {
        ++item;
        return wait_far(sh, &sh.item_full[item & 1], ((item - 1) >> 1) & 1) && sh.item[item & 1].w.pair >= 0;
    };

    if (sh.item[0].w.pair < 0) {
        // nothing: the grid has a CTA for every pair that there might be
    } else if (warp >= 4) {
        // (Sixteen of twenty warps run this, so it comes before the other roles in the code: behind
        // them 900 and 1000 queries x 16 heads behind 7001 keys took 139 us, not 133.6, and 8192 x 32
        // heads 490, not 477, whenever the roles before it had grown.)
        // ---- softmax: two threads a row, 64 of a tile's 128 keys each.  (With one thread a row
        // the chain scores - weights - products of a tile took longer than the tensor cores
        // need for both tiles.)
        const int t = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1, r = (warp & 3) * 32 + lane;
        const uint32_t lane_bits = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_t = tmem + lane_bits + S_COL + t * 128, o_t = tmem + lane_bits + O_COL + t * 128;
        const int pair_bar = 1 + t * 4 + (warp & 3);
        // this thread's value for the row's other thread, and the other's
        const auto swap = [&](float v) {
            sh.other[t][half][r] = v;
            asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory");
            return sh.other[t][half ^ 1][r];
        };
        for (uint32_t item = 0;; ++item) {
            // (what only the pair's end needs stays in shared memory meanwhile)
            const volatile Item &my = sh.item[item & 1];
            int nt, tail, limit;  // limit: keys that this row sees
            {
                const Work w = {0, my.w.nq, 0, my.w.nk, my.w.pair, 0};
                const Extent e(w);
                nt = e.tiles(t);
                tail = e.last() == t ? e.tail() : -1;  // the tile whose values are to be cleared
                limit = e.row0 + t * TM + r + w.nk - w.nq + 1;
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
                    // value rows behind the sequence's last key: whatever follows there must not
                    // meet the zero weights.  (The barrier's fill before this one is used up by
                    // now, so the phase is this fill's.)
                    const uint32_t g = my.g0 + tail;
                    wait(sh, &sh.v_full[g & 1], (g >> 1) & 1);
                    const int z0 = my.w.nk - tail * TN, first = my.slot0 + (tail % Z::SLOTS) * Z::TILE;
#pragma unroll
                    for (int c = KC; c < KC + VC; ++c) {
                        const uint32_t v = ring + (first + c) % Z::SLOTS * CHUNK + z0 * 128;
                        for (int i = half * 128 + r; i < (TN - z0) * 8; i += 256)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(v + i * 16), "r"(0)
                                         : "memory");
                    }
                    fence_async_smem();
                    mbar_arrive(&sh.v_clean);
                }
                tmem_wait_ld();
                if (__builtin_expect(j * TN + TN > limit - r, 0)) {  // more than every row sees
                    const int seen = limit - j * TN - half * 64;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        if (i >= seen) x[0][i] = 0xFF800000u;
                        if (i + 32 >= seen) x[1][i] = 0xFF800000u;
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
                    for (int c = half * (VC * 32); c < (half + 1) * (VC * 32); c += 16) {
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
            const int row = my.w.pair * 2 * TM + t * TM + r, head = my.w.head;
            const bool real = row < my.w.nq;
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // (zero: nothing was seen; NaN stays)
            const int64_t tok = my.w.q0 + row;
            if (real && half == 0 && p.lse)
                p.lse[tok * p.Hq + head] = l == 0.0f ? -INFINITY : (m_ref + log2f(l)) * LN2;
            uint16_t *dst = p.out + tok * p.out_tok + head * p.out_head + half * (VC * 32);
            // 32 bytes a store, a whole sector, where the rows allow it
            const bool sectors = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;
#pragma unroll
            for (int c = 0; c < VC; ++c) {
                uint32_t o[32] = {};
                if (nt > 0) {
                    tmem_ld32(o_t + half * (VC * 32) + 32 * c, o);
                    tmem_wait_ld();
                }
                if (!real) continue;
#pragma unroll
                for (int v = 0; v < 2; ++v) {
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
            // The next pair's products overwrite this output once its first weights are there,
            // which come after these reads.
            tc_fence_before();
            __syncwarp();  // the whole warp is done with the item
            if (lane == 0) mbar_arrive(&sh.item_free[item & 1]);
            if (!all_say<64>(next_item(item), pair_bar)) break;
        }
    } else {
        if (warp == 0) {
            if (elect_one()) {
                // ---- producer
                // The ring holds at most two tiles' chunks, so a slot's last use was in one of
                // the two tiles before; what was waited for once is not waited for again.
                // Tiles are numbered through all pairs of the CTA.
                int64_t j = 0, k_done = -1, v_done = -1;
                int slot = 0, q_uses[2] = {0, 0};
                for (uint32_t item = 0;; ++item) {
                    const Work my = sh.item[item & 1].w;
                    const Extent x(my);
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        if (x.tiles(t) > 0) {
                            if (q_uses[t] > 0 && !wait(sh, &sh.q_free[t], (q_uses[t] - 1) & 1)) break;
                            ++q_uses[t];
                            mbar_expect_tx(&sh.q_full[t], KC * CHUNK);
                            for (int c = 0; c < KC; ++c)
                                tma_load_3d(q_s + (t * KC + c) * CHUNK, &mq, c * 64, my.head,
                                            my.q0 + x.row0 + t * TM, &sh.q_full[t]);
                        }
                    for (int i = 0; i < x.n && !sh.abort; ++i, ++j) {
#pragma unroll
                        for (int c = 0; c < Z::TILE; ++c) {
                            constexpr int TILE = Z::TILE;
                            // the chunk there before, and how many tiles ago
                            const int was = c - Z::SLOTS + 2 * TILE;
                            const int64_t wj = j - (was < TILE ? 2 : was < 2 * TILE ? 1 : 0);
                            if (wj >= 0) {
                                const bool keys = was % TILE < KC;
                                int64_t &done = keys ? k_done : v_done;
                                if (wj > done) {
                                    if (!wait(sh, keys ? &sh.k_free[wj & 1] : &sh.v_free[wj & 1], (wj >> 1) & 1))
                                        break;
                                    done = wj;
                                }
                            }
                            uint64_t *bar = c < KC ? &sh.k_full[j & 1] : &sh.v_full[j & 1];
                            if (c == 0) mbar_expect_tx(bar, KC * CHUNK);
                            if (c == KC) mbar_expect_tx(bar, VC * CHUNK);
                            const uint32_t dst = ring + slot * CHUNK;
                            if (c == KC - 1)
                                tma_load_3d(dst, &mrot, 0, 0, my.k0 + i * TN, bar);
                            else
                                tma_load_3d(dst, &mkv, c < KC ? c * 64 : p.N + (c - KC) * 64, my.head,
                                            my.k0 + i * TN, bar);
                            slot = Z::behind(slot, 1);
                        }
                    }
                    // All that this pair needs is on its way, a tile or two before it is used:
                    // the time to ask for more.  (One, two or five tiles earlier, when work may
                    // go to a CTA that will be free later than another: 8 x 800 tokens x 32
                    // heads 93 -> 94.5, 96, 98; by the issuer at its last tile, 99 us.)
                    mbar_arrive(&sh.near_end);
                    mbar_arrive(&sh.item_free[item & 1]);
                    if (sh.abort || !next_item(item)) break;
                }
                if (sh.abort) {
                    // let the copies in flight land: the last two tiles' and the queries' (a
                    // fill that was cut off never completes: its wait runs to the limit)
                    for (int64_t i = j > 2 ? j - 2 : 0; i < j; ++i) {
                        wait_out(&sh.k_full[i & 1], (i >> 1) & 1);
                        wait_out(&sh.v_full[i & 1], (i >> 1) & 1);
                    }
                    for (int t = 0; t < 2; ++t)
                        if (q_uses[t] > 0) wait_out(&sh.q_full[t], (q_uses[t] - 1) & 1);
                }
            }
        } else if (warp == 1) {
            if (elect_one()) {
                // ---- MMA issuer: a tile's products, then its next scores, in turn
                constexpr uint32_t id_s = idesc_of<T>(TM, TN, false);
                constexpr uint32_t id_o = idesc_of<T>(TM, VC * 64, true), id_o64 = idesc_of<T>(TM, 64, true);
                const uint64_t qd = smem_desc_sw128(q_s), kd = smem_desc_sw128(ring);
                const uint64_t vd = smem_desc_rows_k(ring, CHUNK);
                const auto scores = [&](int slot, int t) {
                    const uint32_t d = tmem + S_COL + t * 128;
                    const uint64_t a = qd + t * (KC * (CHUNK >> 4));
#pragma unroll
                    for (int c = 0; c < KC; ++c) {
                        const uint64_t b = kd + Z::behind(slot, c) * (CHUNK >> 4);
                        if (c < KC - 1 || p.R == 64) {
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                mma_bf16(d, a + c * (CHUNK >> 4) + 2 * u, b + 2 * u, id_s, (c | u) != 0);
                        } else {  // the rotated chunk's columns beyond R are zeros: not worth a step
                            for (int u = 0; u < p.R / 16; ++u)
                                mma_bf16(d, a + c * (CHUNK >> 4) + 2 * u, b + 2 * u, id_s, 1);
                        }
                    }
                    mma_commit(&sh.s_full[t]);
                };
                const auto products = [&](int slot, int t, int j) {
                    const uint32_t a = tmem + S_COL + t * 128, d = tmem + O_COL + t * 128;
                    const uint64_t b = vd + slot * (CHUNK >> 4);
                    if (VC == 1 || slot + 1 < Z::SLOTS) {
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            mma_ts(d, a + 8 * u, b + u * (2048 >> 4), id_o, (j | u) != 0);
                    } else {  // the chunks lie at the ring's two ends
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            mma_ts(d, a + 8 * u, b + u * (2048 >> 4), id_o64, (j | u) != 0);
                            mma_ts(d + 64, a + 8 * u, vd + u * (2048 >> 4), id_o64, (j | u) != 0);
                        }
                    }
                };
                // the slot of the next tile's keys; the tile's number through all pairs, and the
                // numbers of tiles, pairs and cleared tails so far, as far as parities go
                int k = 0;
                uint32_t g = 0, q_uses[2] = {0, 0}, p_uses[2] = {0, 0}, tails = 0;
                for (uint32_t item = 0;; ++item) {
                    const Work my = sh.item[item & 1].w;
                    const Extent x(my);
                    const int last = x.last(), tail = x.tail();
                    if (x.n > 0) {
                        if (!wait(sh, &sh.k_full[g & 1], (g >> 1) & 1)) break;
#pragma unroll
                        for (int t = 0; t < 2; ++t)
                            if (x.tiles(t) > 0) {
                                if (!wait(sh, &sh.q_full[t], q_uses[t] & 1)) break;
                                ++q_uses[t];
                                tc_fence_after();
                                scores(k, t);
                                if (x.tiles(t) == 1) mma_commit(&sh.q_free[t]);
                            }
                        mma_commit(&sh.k_free[g & 1]);
                    }
                    for (int j = 0; j < x.n && !sh.abort; ++j, ++g) {
                        const int v = Z::behind(k, KC);
                        k = Z::behind(v, VC);
                        if (!wait(sh, &sh.v_full[g & 1], (g >> 1) & 1)) break;
                        bool keys = false;  // tile j + 1's have been waited for
                        if (j == tail && !wait(sh, &sh.v_clean, tails++ & 1)) break;
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const int nt = x.tiles(t);
                            if (j >= nt) continue;
                            if (!wait(sh, &sh.p_ready[t], p_uses[t]++ & 1)) break;
                            tc_fence_after();
                            products(v, t, j);
                            if (t == last) mma_commit(&sh.v_free[g & 1]);
                            if (j + 1 == nt) mma_commit(&sh.o_done[t]);
                            if (j + 1 < nt) {
                                if (!keys && !wait(sh, &sh.k_full[(g + 1) & 1], ((g + 1) >> 1) & 1)) break;
                                keys = true;
                                scores(k, t);
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
            // ---- the next work: that of a CTA which has not started yet, so that its queries
            // and keys are on their way while this CTA finishes what it has.  (A CTA a pair
            // spent some 11,000 cycles on its start and its end; so 8 x 800 tokens x 32 heads
            // took 126 us, not 93, and 8192 x 32 heads 472, not 442.)
            Item it = sh.item[0];
            // Request number n: the CTA given, or -1; false if the answer did not come.  The warp
            // decides together, since what follows has full-warp operations; and all lanes have
            // read an answer before the next request lets another be written over it.
            const auto ask = [&](uint32_t n, int &cta) {
                if (lane == 0) {
                    mbar_expect_tx(&sh.answer, sizeof(uint4));
                    ask_for_work(&sh.taken, &sh.answer);
                }
                __syncwarp();
                if (!__all_sync(0xFFFFFFFFu, wait_long(sh, &sh.answer, n & 1))) {
                    wait_out(&sh.answer, n & 1);
                    return false;
                }
                cta = work_given(&sh.taken);
                fence_async_smem();
                __syncwarp();
                return true;
            };
            uint32_t asked = 0;
            for (uint32_t item = 0;; ++item) {
                if (!__all_sync(0xFFFFFFFFu, wait_far(sh, &sh.near_end, item & 1))) break;
                const Extent was(it.w);
                it.g0 += was.n;
                it.slot0 = (it.slot0 + (was.n % Z::SLOTS) * Z::TILE) % Z::SLOTS;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    it.met[t] += was.tiles(t);
                    it.outputs[t] += was.tiles(t) > 0;
                }
                // CTAs without work are among those that have not started (nothing says in which
                // order they are handed out): the next one with work, or the end of them all
                it.w.pair = -1;
                bool there;
                int cta = 0;
                while ((there = ask(asked++, cta)) && cta >= 0) {
                    it.w = work_of(cta);
                    if (it.w.pair >= 0) break;
                }
                if (!there) break;
                // the item before this slot's last is left behind by all (and there is no more work
                // for a CTA that leaves)
                if (!__all_sync(0xFFFFFFFFu, (item == 0 || wait_long(sh, &sh.item_free[(item - 1) & 1],
                                                                     ((item - 1) >> 1) & 1)) &&
                                                 !sh.abort))
                    break;
                if (lane == 0) {
                    sh.item[(item + 1) & 1] = it;
                    mbar_arrive(&sh.item_full[(item + 1) & 1]);
                }
                const Work w = it.w;
                if (w.pair < 0) break;
                if (elect_one()) {
                    const Extent x(w);
                    for (int t = 0; t < 2; ++t)
                        for (int c = 0; c < KC && x.tiles(t) > 0; ++c)
                            tma_prefetch_3d(&mq, c * 64, w.head, w.q0 + x.row0 + t * TM);
                    for (int c = 0; c < KC + VC && x.n > 0; ++c)
                        if (c != KC - 1)
                            tma_prefetch_3d(&mkv, c < KC ? c * 64 : p.N + (c - KC) * 64, w.head, w.k0);
                }
                __syncwarp();
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && sh.abort && p.status) atomicOr(p.status, MTPSPEC_STATUS_TIMEOUT);
    if (warp == 3) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(TMEM_COLS)
                     : "memory");
    }
}

// Diagnostic of the bounded waits: on a barrier of two arrivals that got one, each form must give
// up after `limit` polls and raise the abort flag; and of two warps of which one's wait completed,
// neither goes on.  If any does otherwise, the timeout is taken out of the status word.
__global__ void k_wait_selftest(uint32_t limit, int32_t *status) {
    __shared__ Shared sh;
    uint64_t *never = &sh.item_full[0], *done = &sh.item_full[1];
    if (threadIdx.x == 0) {
        mbar_init(never, 2);
        mbar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        mbar_arrive(never);
        mbar_arrive(done);
    }
    bool ok = true;
    for (int form = 0; form < 4; ++form) {
        __syncthreads();
        if (threadIdx.x == 0) sh.abort = 0;
        __syncthreads();
        bool got;
        if (form == 3) {  // one warp's next item is there, the other's is not
            const int half = threadIdx.x >> 5;
            const bool there = wait_far(sh, half ? never : done, 0, limit);
            ok &= there == (half == 0);
            got = all_say<64>(there, 1);
        } else {
            got = form == 0 ? wait(sh, never, 0, limit)
                  : form == 1 ? wait_long(sh, never, 0, limit) : wait_far(sh, never, 0, limit);
        }
        __syncthreads();
        ok &= !got && sh.abort;
    }
    if (!ok) atomicAnd(status, ~MTPSPEC_STATUS_TIMEOUT);
}

template <typename T, int KC, int VC>
cudaError_t launch(const CUtensorMap &mq, const CUtensorMap &mkv, const CUtensorMap &mrot,
                   const Params &p, cudaStream_t stream) {
    constexpr int smem = Sizes<KC, VC>::SMEM;
    static AttrCache attr;
    cudaError_t e = ensure_attr(k_latent_prefill<T, KC, VC>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem, attr);
    if (e != cudaSuccess) return e;
    const unsigned grid = static_cast<unsigned>(p.ranks) * p.Hq;
    k_latent_prefill<T, KC, VC><<<grid, NTHREADS, smem, stream>>>(mq, mkv, mrot, p);
    e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

template <typename T>
cudaError_t pick(const CUtensorMap &mq, const CUtensorMap &mkv, const CUtensorMap &mrot,
                 const Params &p, cudaStream_t s) {
    if (p.N == 128)
        return p.V == 128 ? launch<T, 3, 2>(mq, mkv, mrot, p, s) : launch<T, 3, 1>(mq, mkv, mrot, p, s);
    return p.V == 128 ? launch<T, 2, 2>(mq, mkv, mrot, p, s) : launch<T, 2, 1>(mq, mkv, mrot, p, s);
}

// A map of [tokens, heads, cols] 16-bit values, in boxes of 128 tokens x 64 columns of a head.
bool token_map(CUtensorMap *m, const uint16_t *ptr, int64_t tokens, int64_t heads, int64_t cols,
               int64_t tok_stride, int64_t head_stride) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    // an axis of one element may come with any stride
    if (heads == 1) head_stride = cols + (-cols & 7);
    if (tokens == 1) tok_stride = head_stride * heads;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(heads),
                          static_cast<cuuint64_t>(tokens)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_stride) * 2,
                             static_cast<cuuint64_t>(tok_stride) * 2};
    cuuint32_t box[3] = {64, 1, 128};
    cuuint32_t es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(ptr), dims, strides, box,
              es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace lpf

cudaError_t run_wait_selftest_latent_prefill(uint32_t limit, int32_t *status, cudaStream_t stream) {
    lpf::k_wait_selftest<<<1, 64, 0, stream>>>(limit, status);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

cudaError_t run_latent_prefill(const LatentPrefillArgs &a, int dtype, cudaStream_t stream) {
    CUtensorMap mq, mkv, mrot;
    if (!lpf::token_map(&mq, a.q, a.Tq, a.Hq, a.N + a.R, a.q_tok, a.q_head) ||
        !lpf::token_map(&mkv, a.kv, a.Tk, a.Hq, a.N + a.V, a.kv_tok, a.kv_head) ||
        !lpf::token_map(&mrot, a.rot, a.Tk, 1, a.R, a.rot_stride, a.R))
        return cudaErrorInvalidValue;
    lpf::Params p = {};
    p.cu_q = a.cu_q;
    p.cu_k = a.cu_k;
    p.B = static_cast<int>(a.B);
    p.Tq = static_cast<int>(a.Tq);
    p.Tk = static_cast<int>(a.Tk);
    p.Hq = a.Hq;
    p.N = a.N;
    p.R = a.R;
    p.V = a.V;
    p.ranks = static_cast<int>((a.Tq + 2 * lpf::TM - 1) / (2 * lpf::TM) + a.B - 1);
    p.scale2 = a.scale * lpf::LOG2E;
    p.out = a.out;
    p.out_tok = a.out_tok;
    p.out_head = a.out_head;
    p.lse = a.lse;
    p.status = a.status;
    return dtype == MTPSPEC_BF16 ? lpf::pick<Bf16>(mq, mkv, mrot, p, stream)
                                 : lpf::pick<F16>(mq, mkv, mrot, p, stream);
}

}  // namespace mtpspec
