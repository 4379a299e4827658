// Attention over the paged latent cache in the absorbed form: every head's query meets the
// cache rows themselves (L latent values and R rotated ones), and the output is the weighted
// sum of the rows' latents.
//
// One pass over the keys with the running maximum and sum of a softmax.  The rows of a
// sequence's (token, head) pairs are cut into tiles of 64, the keys into tiles of 64; a unit
// is one row tile against all keys of its sequence.
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
constexpr int MAX_STAGES = 4;
constexpr int MAX_GROUPS = 4;     // the rotated chunk, then pieces of 256, 128 and 64 columns
constexpr int MAX_BOXES = 8;      // boxes of a tile's chunk: pages of at least eight rows
constexpr int RING = 2;           // tiles whose boxes are known: the current and the next
constexpr int NTHREADS = 192;     // warp 0 TMA, warp 1 MMA and TMEM, warps 2-5 softmax
constexpr int SOFTMAX0 = 64;      // the first softmax thread
constexpr int GRID = 152;         // one CTA per SM of a GB300
constexpr float LAZY = 8.0f;      // the running maximum may lag by a factor of 2^8
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr uint32_t POLL_LIMIT = 1u << 25;  // polls of some 20 ns: ~1 s
constexpr int S_COL = 256;        // TMEM columns: output 0 .. L/2 - 1, scores 2 x 32 from here
constexpr uint32_t TMEM_COLS = 512;

struct Params {
    const uint16_t *q;
    int64_t q_row, q_tok, q_head;
    const int32_t *block_table, *kv_len;
    int64_t max_pages;
    int num_pages, page_size, box_rows;
    int B, T, Hq, L, R, stages;
    int mtiles;          // row tiles of a sequence
    int gs, mgroups;     // CTAs that walk the same keys, one row tile each; such groups a sequence
    int groups;          // groups of CTAs in the grid
    float scale2;  // scale * log2(e), above 0
    uint16_t *out;
    int64_t out_row, out_tok, out_head;
    float *lse;
    int2 *plan;      // [B * mgroups]: first and last group of a unit
    float *part;     // [2 * GRID][rows][L] fp32, normalised partial outputs
    float *part_lse; // [2 * GRID][rows], base 2
    int rows_cap;    // rows of a partial: min(64, T * Hq)
    int32_t *status;
};

__device__ __forceinline__ int row_len(const Params &p, int b) {
    const int64_t cap = p.max_pages * p.page_size;
    const int n = p.kv_len[b];
    return n < 0 ? 0 : static_cast<int>(n < cap ? n : cap);
}
__device__ __forceinline__ int row_tiles(const Params &p, int b) {
    return (row_len(p, b) + TN - 1) / TN;
}

// How many of the groups take part, and the first tile of one of them: an even cut of all
// units' tiles laid end to end.
__device__ __forceinline__ int active_groups(const Params &p, int64_t total) {
    return static_cast<int>(total < p.groups ? (total > 0 ? total : 1) : p.groups);
}
__device__ __forceinline__ int64_t first_tile(int64_t total, int active, int g) {
    return total * g / active;
}
__device__ __forceinline__ int owner(int64_t total, int active, int64_t tile) {
    return static_cast<int>(((tile + 1) * active - 1) / total);
}

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
                nt = row_tiles(p, b);
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
        len = row_len(p, ib);
        return true;
    }
};

struct __align__(16) Shared {
    uint64_t full[MAX_STAGES][MAX_GROUPS], empty[MAX_STAGES][MAX_GROUPS];
    uint64_t s_full[2], p_ready, pv_done, q_ready, o_empty;
    uint64_t drained;
    float xm[2][4][32];
    int2 box[RING][MAX_BOXES];
    int64_t scan[NTHREADS / 32];
    int64_t total;
    int start_b, start_mg, start_off, start_nt;
    uint32_t tmem;
    volatile int abort;
};

constexpr int SMEM_MAX = 232448;                                        // 227 KB a CTA
constexpr int SMEM_EXTRA = static_cast<int>(sizeof(Shared)) + 1024;    // and the alignment

// A bounded wait; once any wait of the CTA has given up, the others return at once, and the
// roles run to their ends without touching what they could not wait for.
__device__ __forceinline__ bool wait(Shared &sh, uint64_t *bar, uint32_t parity) {
    for (uint32_t it = 0; it < POLL_LIMIT; ++it) {
        if (mbar_poll(bar, parity)) return true;
        if (sh.abort) return false;
    }
    sh.abort = 1;
    return false;
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
// The descriptor of a tile whose 64-column chunks lie CHUNK bytes apart and whose rows are
// the products' K axis (the "MN-major" form): 8-row groups every 1024 bytes.
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

// The output's columns in pieces of 256, 128 and 64 (the widths of the folded accumulator).
__device__ __forceinline__ int piece_width(int left) {
    return left >= 256 ? 256 : (left >= 128 ? 128 : 64);
}

template <typename T>
__global__ void __launch_bounds__(NTHREADS, 1)
k_latent_attn(const __grid_constant__ CUtensorMap map, const Params p) {
    extern __shared__ uint8_t smem_dyn[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~static_cast<uintptr_t>(1023));
    const int nchunks = p.L / 64 + 1;
    const uint32_t base = smem_addr(smem);
    const uint32_t q_s = base, p_s = base + nchunks * CHUNK, kv_s = p_s + CHUNK;
    const int stage_bytes = nchunks * CHUNK;
    Shared &sh = *reinterpret_cast<Shared *>(smem + (1 + p.stages) * stage_bytes + CHUNK);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < MAX_STAGES * MAX_GROUPS; ++i) {
            mbar_init(&sh.full[0][0] + i, 1);
            mbar_init(&sh.empty[0][0] + i, 1);
        }
        mbar_init(&sh.s_full[0], 1);
        mbar_init(&sh.s_full[1], 1);
        mbar_init(&sh.p_ready, 128);
        mbar_init(&sh.pv_done, 1);
        mbar_init(&sh.q_ready, 128);
        mbar_init(&sh.o_empty, 128);
        mbar_init(&sh.drained, 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&map);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(&sh.tmem)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // ---- where this CTA starts: a scan of the rows' tiles, one run of rows a thread
    const int per = (p.B + NTHREADS - 1) / NTHREADS;
    const int r0 = min(p.B, static_cast<int>(threadIdx.x) * per), r1 = min(p.B, r0 + per);
    int64_t sum = 0;
    for (int b = r0; b < r1; ++b) sum += static_cast<int64_t>(row_tiles(p, b)) * p.mgroups;
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) sh.scan[warp] = incl;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int64_t before = 0, total = 0;
    for (int w = 0; w < NTHREADS / 32; ++w) {
        if (w < warp) before += sh.scan[w];
        total += sh.scan[w];
    }
    const int active = active_groups(p, total);
    const int cta = blockIdx.x, group = cta / p.gs;
    const int64_t t0 = group < active ? first_tile(total, active, group) : total;
    const int64_t t1 = group < active ? first_tile(total, active, group + 1) : total;
    int64_t at = before + incl - sum;
    if (t0 < t1 && at <= t0 && t0 < at + sum) {
        int b = r0;
        for (;; ++b) {
            const int64_t n = static_cast<int64_t>(row_tiles(p, b)) * p.mgroups;
            if (t0 < at + n) break;
            at += n;
        }
        sh.start_b = b;
        sh.start_nt = row_tiles(p, b);
        sh.start_mg = static_cast<int>((t0 - at) / sh.start_nt);
        sh.start_off = static_cast<int>((t0 - at) % sh.start_nt);
    }
    __syncthreads();
    const uint32_t tmem = sh.tmem;
    Walk w;
    w.left = t1 - t0;
    w.lane = cta - group * p.gs;
    if (w.left > 0) {
        w.b = sh.start_b;
        w.mg = sh.start_mg;
        w.off = sh.start_off;
        w.nt = sh.start_nt;
    }

    if (warp == 0) {
        if (elect_one()) {
            // ---- producer: a tile's chunks group by group, in boxes that stay within a
            // page.  Each box's page is looked up a tile ahead.
            const int boxes = TN / p.box_rows;
            int g = 0, k = 0, s = 0;
            uint32_t ph = 1;  // phase of stage s's release
            while (!sh.abort && w.next(p)) {
                const int32_t *table = p.block_table + w.ib * p.max_pages;
                int f = w.i0;  // the next tile to look up
                for (int tile = w.i0; tile < w.i1; ++tile, ++g) {
                    for (; f < w.i1 && f < tile + RING; ++f) {
                        int key = f * TN, pi = key / p.page_size, row = key - pi * p.page_size;
                        int page[MAX_BOXES], off[MAX_BOXES];
#pragma unroll
                        for (int i = 0; i < MAX_BOXES; ++i) {
                            page[i] = p.num_pages;  // beyond the last page: TMA fills zeros
                            off[i] = row;
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
#pragma unroll
                        for (int i = 0; i < MAX_BOXES; ++i) {
                            if (i >= boxes) break;
                            if (static_cast<unsigned>(page[i]) > static_cast<unsigned>(p.num_pages) ||
                                (page[i] == p.num_pages && f * TN + i * p.box_rows < w.len)) {
                                page[i] = p.num_pages;
                                if (p.status) atomicOr(p.status, MTPSPEC_STATUS_BAD_PARAM);
                            }
                            sh.box[f % RING][i] = make_int2(page[i], off[i]);
                        }
                    }
                    int o = 0;
                    for (k = 0; k < MAX_GROUPS; ++k) {
                        // group 0: the rotated chunk; group k: the output's k-th piece
                        if (k > 0 && o >= p.L) break;
                        const int c0 = k == 0 ? nchunks - 1 : o / 64;
                        const int n = k == 0 ? 1 : piece_width(p.L - o) / 64;
                        if (k > 0) o += n * 64;
                        if (!wait(sh, &sh.empty[s][k], ph)) break;
                        mbar_expect_tx(&sh.full[s][k], n * CHUNK);
                        uint32_t dst = kv_s + s * stage_bytes + c0 * CHUNK;
#pragma unroll
                        for (int i = 0; i < MAX_BOXES; ++i) {
                            if (i >= boxes) break;
                            const int2 x = sh.box[tile % RING][i];
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                if (c < n)
                                    tma_load_3d(dst + c * CHUNK, &map, (c0 + c) * 64, x.y, x.x,
                                                &sh.full[s][k]);
                            dst += p.box_rows * 128;
                        }
                    }
                    if (sh.abort) break;
                    if (++s == p.stages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            // after an abort, let the copies in flight land (the last fill of each barrier)
            if (sh.abort)
                for (int j = 0; j < p.stages; ++j)
                    for (int i = 0; i < MAX_GROUPS; ++i) {
                        const int n = (g + p.stages - 1 - j) / p.stages + (j == s && i < k);
                        for (uint32_t it = 0; n > 0 && it < WAIT_LIMIT; ++it)
                            if (mbar_test(&sh.full[j][i], (n - 1) & 1)) break;
                    }
        }
    } else if (warp == 1) {
        if (elect_one()) {
            // ---- MMA issuer.  Two kinds of work wait for different things: the scores of
            // tile a for its chunks, the products of tile b for its weights.  Whichever is
            // there is issued, the products first, since they free the stage.
            constexpr uint32_t id_qk = idesc_of<T>(TN, false);
            const uint64_t qd = smem_desc_sw128(q_s), pd = smem_desc_sw128(p_s);
            int item = 0;
            int sa = 0, sb = 0;           // the stages of tiles a and b
            uint32_t pa = 0, par = 0;     // phase of stage sa; parity of tile a's number
            int ahead = 0;                // tiles whose scores are issued, products not
            uint32_t pb = 0, idle = 0;    // parity of tile b's number
            bool first = true;            // tile b is the item's first
            auto products = [&]() {       // false: not ready
                if (ahead == 0 || !mbar_poll(&sh.p_ready, pb)) {
                    if (++idle > POLL_LIMIT) sh.abort = 1;
                    return false;
                }
                if (first && item > 0 && !wait(sh, &sh.o_empty, (item - 1) & 1)) return false;
                tc_fence_after();
                const uint64_t vd0 = smem_desc_rows_k(kv_s + sb * stage_bytes);
                for (int c = 0, k = 1; c < p.L; ++k) {
                    const int n = piece_width(p.L - c);
                    const uint32_t id = idesc_of<T>(n, true);
                    const uint64_t vd = vd0 + (c / 64) * (CHUNK >> 4);
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        mma_ws(tmem + c / 2, pd + 2 * u, vd + u * (2048 >> 4), id, !first || u > 0);
                    mma_commit(&sh.empty[sb][k]);
                    c += n;
                }
                mma_commit(&sh.pv_done);
                if (++sb == p.stages) sb = 0;
                pb ^= 1;
                --ahead;
                first = false;
                idle = 0;
                return true;
            };
            while (!sh.abort && w.next(p)) {
                if (!wait(sh, &sh.q_ready, item & 1)) break;
                tc_fence_after();
                first = true;
                for (int tile = w.i0; tile < w.i1 && !sh.abort; ++tile) {
                    while (ahead > 1 && !sh.abort) products();  // the scores' buffer is free
                    const uint64_t kd0 = smem_desc_sw128(kv_s + sa * stage_bytes);
                    const uint32_t d = tmem + S_COL + par * (TN / 2);
                    int o = 0;
#pragma unroll
                    for (int k = 0; k < MAX_GROUPS; ++k) {
                        if (k > 0 && o >= p.L) break;
                        const int c0 = k == 0 ? nchunks - 1 : o / 64;
                        const int n = k == 0 ? 1 : piece_width(p.L - o) / 64;
                        if (k > 0) o += n * 64;
                        do {
                            products();
                        } while (!mbar_poll(&sh.full[sa][k], pa) && !sh.abort);
                        if (sh.abort) break;
                        idle = 0;
                        tc_fence_after();
                        const uint64_t ad = qd + c0 * (CHUNK >> 4), bd = kd0 + c0 * (CHUNK >> 4);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            if (c >= n) break;
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                mma_ws(d, ad + c * (CHUNK >> 4) + 2 * u, bd + c * (CHUNK >> 4) + 2 * u,
                                       id_qk, (k | c | u) != 0);
                        }
                        if (k == 0) mma_commit(&sh.empty[sa][0]);
                    }
                    mma_commit(&sh.s_full[par]);
                    ++ahead;
                    par ^= 1;
                    if (++sa == p.stages) {
                        sa = 0;
                        pa ^= 1;
                    }
                }
                while (ahead > 0 && !sh.abort) products();
                ++item;
            }
            mma_commit(&sh.drained);
            for (uint32_t it = 0; it < WAIT_LIMIT; ++it)
                if (mbar_test(&sh.drained, 0)) break;
        }
    } else {
        // ---- softmax: a pair of threads a row, 32 of a tile's 64 keys each
        const int wq = warp & 3, half = wq >> 1, r = (wq & 1) * 32 + lane;
        const int tid = threadIdx.x - SOFTMAX0;
        const uint32_t trow = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const int vecs = (p.L + p.R) / 8, vecs_all = nchunks * 8;
        const int rows_all = p.T * p.Hq;
        int g = 0, slot = 0, stage = 0;
        Walk nw = w;  // one item ahead: its queries are loaded before this item's epilogue
        bool more = nw.next(p);
        auto load_q = [&](const Walk &k) {
            // two threads a row, every other vector each; what lies beyond is zero
            const int row = tid >> 1, m = k.imt * TM + row;
            const bool real = m < rows_all;
            const int t = real ? m / p.Hq : 0, h = real ? m - t * p.Hq : 0;
            const uint16_t *src = p.q + (k.ib * p.q_row + t * p.q_tok + h * p.q_head);
            const uint32_t dst = q_s + row * 128;
#pragma unroll 4
            for (int v = tid & 1; v < vecs_all; v += 2) {
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
        while (more) {
            w = nw;
            const int m = w.imt * TM + r;
            const int limit = w.len - (p.T - 1 - min(m, rows_all - 1) / p.Hq);
            const int sure = w.len - (p.T - 1 - (w.imt * TM) / p.Hq);  // the least limit
            float m_ref = -INFINITY, l = 0.0f;
            for (int tile = w.i0; tile < w.i1; ++tile, ++g) {
                wait(sh, &sh.s_full[g & 1], (g >> 1) & 1);
                tc_fence_after();
                uint32_t raw[32];
                tmem_ld32(trow + S_COL + (g & 1) * (TN / 2), raw);
                tmem_wait_ld();
                float x[32], top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(raw[i]);
                if (tile * TN + TN > sure) {
                    const int k0 = tile * TN + half * 32;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (k0 + i >= limit) x[i] = -INFINITY;
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) top4[i & 3] = fmaxf(top4[i & 3], x[i]);
                float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
                sh.xm[slot][wq][lane] = top;
                asm volatile("bar.sync %0, 64;" ::"r"(1 + (wq & 1)) : "memory");
                top = fmaxf(top, sh.xm[slot][wq ^ 2][lane]) * p.scale2;
                slot ^= 1;
                const bool raise = top > m_ref + LAZY;
                const float m_old = m_ref;
                if (raise) m_ref = top;
                const float m_use = m_ref == -INFINITY ? 0.0f : m_ref;
                float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                uint4 weights[4];
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    float e[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        e[u] = ex2(fmaf(x[8 * v + u], p.scale2, -m_use));
                        part[u & 3] += e[u];
                    }
                    weights[v] = float_to_half8<T>(e);
                }
                // the products of the tile before are done: the weights' buffer and the
                // output are free to change
                if (g > 0) wait(sh, &sh.pv_done, (g - 1) & 1);
                if (tile > w.i0 && __any_sync(0xFFFFFFFFu, raise)) {
                    tc_fence_after();
                    const float f = raise ? ex2(m_old - m_ref) : 1.0f;
                    l *= f;
                    for (int c = 0; c < p.L / 2; c += 32) {
                        uint32_t o[32];
                        tmem_ld32(trow + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tmem_st32(trow + c, o);
                    }
                    tmem_wait_st();
                }
                l += (part[0] + part[1]) + (part[2] + part[3]);
                const uint32_t prow = p_s + r * 128;
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                     prow + (((half * 4 + v) ^ (r & 7)) << 4)),
                                 "r"(weights[v].x), "r"(weights[v].y), "r"(weights[v].z),
                                 "r"(weights[v].w)
                                 : "memory");
                if (tile * TN + TN > w.len) {
                    // rows of the tile beyond the sequence: whatever the page holds there
                    // must not meet the zero weights
                    const uint32_t v = kv_s + stage * stage_bytes;
                    const int z0 = w.len - tile * TN;
                    for (int i = tid; i < (TN - z0) * 8 * (p.L / 64); i += 128) {
                        const int c = i / ((TN - z0) * 8), j = i - c * ((TN - z0) * 8);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                         v + c * CHUNK + z0 * 128 + j * 16),
                                     "r"(0)
                                     : "memory");
                    }
                }
                fence_async_smem();
                tc_fence_before();
                mbar_arrive(&sh.p_ready);
                if (++stage == p.stages) stage = 0;
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
            const float inv = l > 0.0f ? 1.0f / l : 0.0f;
            const float lse2 = l > 0.0f ? m_ref + log2f(l) : -INFINITY;
            const int t = m / p.Hq, h = m - t * p.Hq;
            const int64_t prow =
                static_cast<int64_t>(2 * cta + (w.i0 > 0 ? 0 : 1)) * p.rows_cap + r;
            if (real && half == 0) {
                if (!whole)
                    p.part_lse[prow] = lse2;
                else if (p.lse)
                    p.lse[(static_cast<int64_t>(w.ib) * p.T + t) * p.Hq + h] = lse2 * LN2;
            }
            if (tid == 0 && w.i0 == 0 && w.lane == 0) {
                // this item starts its unit: the unit's last tile is int_ - 1 tiles on
                const int64_t last = t1 - w.left - (w.i1 - w.i0) + w.int_ - 1;
                p.plan[static_cast<int64_t>(w.ib) * p.mgroups + w.imt / p.gs] =
                    make_int2(group, owner(total, active, last));
            }
            uint16_t *dst = p.out + w.ib * p.out_row + t * p.out_tok + h * p.out_head;
            float *pdst = p.part + prow * p.L;
            for (int o = 0; o < p.L;) {
                const int n = piece_width(p.L - o);
                for (int c = 0; c < n / 2; c += 32) {
                    uint32_t a[32];
                    tmem_ld32(trow + o / 2 + c, a);
                    tmem_wait_ld();
                    const int col = o + half * (n / 2) + c;
                    if (!real) continue;
                    if (whole) {
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            float f[8];
#pragma unroll
                            for (int u = 0; u < 8; ++u) f[u] = __uint_as_float(a[8 * v + u]) * inv;
                            *reinterpret_cast<uint4 *>(dst + col + 8 * v) = float_to_half8<T>(f);
                        }
                    } else {
#pragma unroll
                        for (int v = 0; v < 8; ++v)
                            *reinterpret_cast<float4 *>(pdst + col + 4 * v) = make_float4(
                                __uint_as_float(a[4 * v]) * inv, __uint_as_float(a[4 * v + 1]) * inv,
                                __uint_as_float(a[4 * v + 2]) * inv, __uint_as_float(a[4 * v + 3]) * inv);
                    }
                }
                o += n;
            }
            tc_fence_before();
            mbar_arrive(&sh.o_empty);
        }
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

// Units cut among CTAs: each row's partial outputs, weighted by their sums, become the
// output.  Rows of empty sequences get zeros.  One warp a row of a unit.
constexpr int JOIN_THREADS = 128;

template <typename T>
__global__ void __launch_bounds__(JOIN_THREADS) k_latent_join(const Params p) {
    pdl_wait_primary();
    const int lane = threadIdx.x & 31;
    const int rows_all = p.T * p.Hq;
    const int64_t m_all = static_cast<int64_t>(blockIdx.x) * (JOIN_THREADS / 32) + (threadIdx.x >> 5);
    const int b = static_cast<int>(m_all / rows_all);
    if (b >= p.B) return;
    const int m = static_cast<int>(m_all - static_cast<int64_t>(b) * rows_all);
    const int t = m / p.Hq, h = m - t * p.Hq;
    const int n = p.kv_len[b];
    if (p.status && m == 0 && lane == 0 && (n < 0 || n > p.max_pages * p.page_size))
        atomicOr(p.status, MTPSPEC_STATUS_BAD_PARAM);
    uint16_t *dst = p.out + b * p.out_row + t * p.out_tok + h * p.out_head;
    if (row_len(p, b) == 0) {
        for (int c = lane * 8; c < p.L; c += 256) *reinterpret_cast<uint4 *>(dst + c) = make_uint4(0, 0, 0, 0);
        if (p.lse && lane == 0) p.lse[m_all] = -INFINITY;
        return;
    }
    const int mt = m / TM, mg = mt / p.gs, r = m - mt * TM;
    const int2 span = p.plan[static_cast<int64_t>(b) * p.mgroups + mg];
    if (span.x == span.y) return;
    // the partial of a group: its second slot where the unit starts, else its first
    const auto part_row = [&](int g) {
        const int64_t cta = static_cast<int64_t>(g) * p.gs + (mt - mg * p.gs);
        return (2 * cta + (g == span.x)) * p.rows_cap + r;
    };
    float top = -INFINITY;
    for (int c = span.x + lane; c <= span.y; c += 32)
        top = fmaxf(top, p.part_lse[part_row(c)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    float acc[2][8] = {}, sum = 0.0f;
    if (top > -INFINITY)
        for (int c = span.x; c <= span.y; ++c) {
            const int64_t row = part_row(c);
            const float wgt = exp2f(p.part_lse[row] - top);
            sum += wgt;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int col = lane * 8 + 256 * k;
                if (col < p.L) {
                    const float4 v0 = *reinterpret_cast<const float4 *>(p.part + row * p.L + col);
                    const float4 v1 = *reinterpret_cast<const float4 *>(p.part + row * p.L + col + 4);
                    acc[k][0] += wgt * v0.x;
                    acc[k][1] += wgt * v0.y;
                    acc[k][2] += wgt * v0.z;
                    acc[k][3] += wgt * v0.w;
                    acc[k][4] += wgt * v1.x;
                    acc[k][5] += wgt * v1.y;
                    acc[k][6] += wgt * v1.z;
                    acc[k][7] += wgt * v1.w;
                }
            }
        }
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int col = lane * 8 + 256 * k;
        if (col >= p.L) continue;
#pragma unroll
        for (int u = 0; u < 8; ++u) acc[k][u] *= inv;
        *reinterpret_cast<uint4 *>(dst + col) = float_to_half8<T>(acc[k]);
    }
    if (p.lse && lane == 0) p.lse[m_all] = sum > 0.0f ? (top + log2f(sum)) * LN2 : -INFINITY;
}

size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

struct Layout {
    size_t plan, part, lse, total;
    int mtiles, gs, mgroups, rows_cap;
};
Layout layout(int64_t B, int64_t rows, int32_t L) {
    Layout y;
    y.mtiles = static_cast<int>((rows + TM - 1) / TM);
    // CTAs that share their keys walk them side by side, so that the keys leave HBM once;
    // up to eight, in as even groups as there are
    y.mgroups = (y.mtiles + 7) / 8;
    y.gs = (y.mtiles + y.mgroups - 1) / y.mgroups;
    y.rows_cap = static_cast<int>(std::min<int64_t>(rows, TM));
    y.plan = 0;
    y.part = align256(static_cast<size_t>(B) * y.mgroups * sizeof(int2));
    y.lse = y.part + align256(static_cast<size_t>(2 * GRID) * y.rows_cap * L * 4);
    y.total = y.lse + align256(static_cast<size_t>(2 * GRID) * y.rows_cap * 4);
    return y;
}

template <typename T>
cudaError_t launch(const CUtensorMap &map, const Params &p, cudaStream_t stream) {
    const int smem = (1 + p.stages) * (p.L / 64 + 1) * CHUNK + CHUNK + SMEM_EXTRA;
    static AttrCache attr;
    cudaError_t e = ensure_attr(k_latent_attn<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem, attr);
    if (e != cudaSuccess) return e;
    k_latent_attn<T><<<GRID, NTHREADS, smem, stream>>>(map, p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    count_launches(1);
    const int64_t rows = static_cast<int64_t>(p.B) * p.T * p.Hq;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((rows + JOIN_THREADS / 32 - 1) / (JOIN_THREADS / 32)));
    cfg.blockDim = dim3(JOIN_THREADS);
    cfg.stream = stream;
    cfg.attrs = pdl_attr();
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_latent_join<T>, p);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace lat

size_t latent_attn_workspace_bytes(int64_t B, int32_t T, int32_t Hq, int32_t L) {
    return lat::layout(B, static_cast<int64_t>(T) * Hq, L).total;
}

cudaError_t run_latent_attn(const LatentAttnArgs &a, int dtype, cudaStream_t stream) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    // boxes of the largest power of two (up to a tile) that divides the page: a box never
    // leaves its page, and its rows start at a multiple of eight, the swizzle's period
    const int box = std::min(lat::TN, a.page_size & -a.page_size);
    CUtensorMap map;
    const cuuint64_t W = static_cast<cuuint64_t>(a.L + a.R);
    cuuint64_t dims[3] = {W, static_cast<cuuint64_t>(a.page_size), static_cast<cuuint64_t>(a.num_pages)};
    cuuint64_t strides[2] = {W * 2, static_cast<cuuint64_t>(a.page_stride) * 2};
    cuuint32_t boxes[3] = {64, static_cast<cuuint32_t>(box), 1};
    cuuint32_t es[3] = {1, 1, 1};
    if (fn(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(a.cache), dims, strides,
           boxes, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    const lat::Layout y = lat::layout(a.B, static_cast<int64_t>(a.T) * a.Hq, a.L);
    unsigned char *ws = static_cast<unsigned char *>(a.workspace);
    lat::Params p = {};
    p.q = a.q;
    p.q_row = a.q_row;
    p.q_tok = a.q_tok;
    p.q_head = a.q_head;
    p.block_table = a.block_table;
    p.kv_len = a.kv_len;
    p.max_pages = a.max_pages;
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
    const int stage = (a.L / 64 + 1) * lat::CHUNK;
    p.stages = std::min<int>(lat::MAX_STAGES,
                             (lat::SMEM_MAX - stage - lat::CHUNK - lat::SMEM_EXTRA) / stage);
    p.scale2 = a.scale * lat::LOG2E;
    p.out = a.out;
    p.out_row = a.out_row;
    p.out_tok = a.out_tok;
    p.out_head = a.out_head;
    p.lse = a.lse;
    p.plan = reinterpret_cast<int2 *>(ws + y.plan);
    p.part = reinterpret_cast<float *>(ws + y.part);
    p.part_lse = reinterpret_cast<float *>(ws + y.lse);
    p.rows_cap = y.rows_cap;
    p.status = a.status;
    return dtype == MTPSPEC_BF16 ? lat::launch<Bf16>(map, p, stream) : lat::launch<F16>(map, p, stream);
}

}  // namespace mtpspec
