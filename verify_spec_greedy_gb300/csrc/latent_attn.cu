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
    int4 *plan;      // [GRID]: the unit that starts in a CTA and ends in another: row, row
                     // tile, first and last group; row -1 if there is none
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
    uint64_t full[MAX_STAGES][MAX_GROUPS], empty[MAX_STAGES][MAX_GROUPS];
    uint64_t s_full[2], p_ready, pv_done, q_ready, o_empty;
    uint64_t drained;
    float xm[2][4][32];
    int2 box[RING][MAX_BOXES];
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

    if (warp == 0) {
        if (lane < MAX_STAGES * MAX_GROUPS) {
            mbar_init(&sh.full[0][0] + lane, 1);
            mbar_init(&sh.empty[0][0] + lane, 1);
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
            prefetch_map(&map);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(&sh.tmem)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_wait_primary();
    // ---- where this CTA starts.  Every warp finds it by itself, from a scan of the rows'
    // tiles with a run of rows a lane: no role waits for another's.
    const int per_lane = (p.B + 31) / 32;
    const int r0 = min(p.B, lane * per_lane), r1 = min(p.B, r0 + per_lane);
    int64_t sum = 0;
#pragma unroll 4
    for (int b = r0; b < r1; ++b) sum += static_cast<int64_t>(tiles_of(row_len(p, b))) * p.mgroups;
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
        int b = r0, n = 0, in = 0;
        if (mine)
            for (;; ++b) {
                n = row_len(p, b);
                const int64_t unit_tiles = static_cast<int64_t>(tiles_of(n)) * p.mgroups;
                if (t0 < at + unit_tiles) break;
                at += unit_tiles;
            }
        in = static_cast<int>(t0 - at);  // fewer than 2^31 tiles a row
        const unsigned who = __ballot_sync(0xFFFFFFFFu, mine);
        const int src = who ? __ffs(who) - 1 : 0;
        w.b = __shfl_sync(0xFFFFFFFFu, b, src);
        w.len = __shfl_sync(0xFFFFFFFFu, n, src);
        w.off = __shfl_sync(0xFFFFFFFFu, in, src);
        w.nt = tiles_of(w.len);
        w.mg = 0;
        if (p.mgroups > 1 && w.nt > 0) {
            w.mg = w.off / w.nt;
            w.off -= w.mg * w.nt;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;

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
            pdl_launch_dependents();  // the joining kernel may be set up; it waits for this one
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
        // ---- rows without keys, and lengths out of range, while the first keys are on their way
        for (int b = cta; b < p.B; b += GRID) {
            const int n = p.kv_len[b];
            if (tid == 0 && p.status && (n < 0 || n > p.max_pages * p.page_size))
                atomicOr(p.status, MTPSPEC_STATUS_BAD_PARAM);
            if (row_len(p, b) > 0) continue;
            const int row_vecs = p.L / 8;
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
        int4 cut_unit = make_int4(-1, 0, 0, 0);
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
            if (real && half == 0) {
                if (!whole)
                    p.part_lse[(2 * cta + (w.i0 > 0 ? 0 : 1)) * static_cast<int64_t>(p.rows_cap) + r] =
                        lse2;
                else if (p.lse)
                    p.lse[static_cast<int64_t>(w.ib) * rows_all + m] = lse2 * LN2;
            }
            if (w.i0 == 0 && !whole)  // the unit starts here and goes on in other groups
                cut_unit = make_int4(w.ib, w.imt, group,
                                     cut.owner(t1 - w.left - (w.i1 - w.i0) + w.int_ - 1));
            // A row a thread: stores of 32 bytes, a whole sector each, where the rows allow it
            const int t = m / p.Hq, h = m - t * p.Hq;
            uint16_t *dst = p.out + w.ib * p.out_row + t * p.out_tok + h * p.out_head;
            float *pdst = p.part + ((2 * cta + (w.i0 > 0 ? 0 : 1)) * static_cast<int64_t>(p.rows_cap) + r) * p.L;
            const bool sectors = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;
            uint32_t a[2][32];
            tmem_ld32(trow, a[0]);
            int o = 0, n = piece_width(p.L), c = 0;
#pragma unroll 2
            for (int i = 0; i < p.L / 64; ++i) {
                tmem_wait_ld();
                if (i + 1 < p.L / 64) tmem_ld32(trow + 32 * (i + 1), a[(i + 1) & 1]);
                const int col = o + half * (n / 2) + c;
                c += 32;
                if (c == n / 2) {
                    o += n;
                    n = piece_width(p.L - o);
                    c = 0;
                }
                if (!real) continue;
                float f[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) f[k] = __uint_as_float(a[i & 1][k]) * inv;
                if (whole) {
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        uint32_t x[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) x[k] = T::narrow2(f[16 * v + 2 * k], f[16 * v + 2 * k + 1]);
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
                        for (int k = 0; k < 8; ++k) x[k] = __float_as_uint(f[8 * v + k]);
                        st_global_32B(pdst + col + 8 * v, x);
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(&sh.o_empty);
        }
        if (tid == 0) p.plan[cta] = cut_unit;
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
// output.  A CTA takes one row of the unit that starts in CTA blockIdx.y of the first kernel
// and ends in another group; a thread takes four columns of every part, eight parts in flight.
constexpr int JOIN_THREADS = 128;

template <typename T>
__global__ void __launch_bounds__(JOIN_THREADS) k_latent_join(const Params p) {
    __shared__ float weight[GRID];
    pdl_wait_primary();
    const int4 u = p.plan[blockIdx.y];
    // (what an aborted call left there is checked)
    if (u.x < 0 || u.x >= p.B || u.y < 0 || u.y >= p.mtiles || u.z < 0 || u.w >= p.groups) return;
    const int r = blockIdx.x, m = u.y * TM + r, rows_all = p.T * p.Hq, parts = u.w - u.z + 1;
    if (m >= rows_all || parts < 2) return;
    // a group's partial of this row: the second slot where the unit starts, else the first
    const int lane_cta = u.y % p.gs;
    const auto part_row = [&](int i) {
        const int64_t cta = static_cast<int64_t>(u.z + i) * p.gs + lane_cta;
        return (2 * cta + (i == 0)) * p.rows_cap + r;
    };
    // every warp finds the row's largest sum by itself
    const int lane = threadIdx.x & 31;
    float top = -INFINITY, sum = 0.0f;
    for (int i = lane; i < parts; i += 32) top = fmaxf(top, p.part_lse[part_row(i)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const float ref = top == -INFINITY ? 0.0f : top;
    for (int i = lane; i < parts; i += 32) {
        const float w = exp2f(p.part_lse[part_row(i)] - ref);
        sum += w;
        if (threadIdx.x < 32) weight[i] = w;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    __syncthreads();
    const int col = threadIdx.x * 4;
    if (col < p.L) {
        const float *src = p.part + col;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int i = 0; i < parts; i += 8) {
            float4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (i + k < parts) v[k] = *reinterpret_cast<const float4 *>(src + part_row(i + k) * p.L);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (i + k < parts) {
                    const float w = weight[i + k];
                    acc.x += w * v[k].x;
                    acc.y += w * v[k].y;
                    acc.z += w * v[k].z;
                    acc.w += w * v[k].w;
                }
        }
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
        const int t = m / p.Hq, h = m - t * p.Hq;
        *reinterpret_cast<uint2 *>(p.out + u.x * p.out_row + t * p.out_tok + h * p.out_head + col) =
            make_uint2(T::narrow2(acc.x * inv, acc.y * inv), T::narrow2(acc.z * inv, acc.w * inv));
    }
    if (p.lse && threadIdx.x == 0)
        p.lse[static_cast<int64_t>(u.x) * rows_all + m] = sum > 0.0f ? (top + log2f(sum)) * LN2 : -INFINITY;
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
    y.part = align256(GRID * sizeof(int4));
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(GRID);
    cfg.blockDim = dim3(NTHREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = pdl_attr();  // set up beside the end of whatever the stream runs before
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_latent_attn<T>, map, p);
    if (e != cudaSuccess) return e;
    count_launches(1);
    cfg.gridDim = dim3(p.rows_cap, p.groups * p.gs);
    cfg.blockDim = dim3(JOIN_THREADS);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, k_latent_join<T>, p);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace lat

size_t latent_attn_workspace_bytes(int64_t B, int32_t T, int32_t Hq, int32_t L) {
    (void)B;
    return lat::layout(static_cast<int64_t>(T) * Hq, L).total;
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
    p.plan = reinterpret_cast<int4 *>(ws + y.plan);
    p.part = reinterpret_cast<float *>(ws + y.part);
    p.part_lse = reinterpret_cast<float *>(ws + y.lse);
    p.rows_cap = y.rows_cap;
    p.status = a.status;
    return dtype == MTPSPEC_BF16 ? lat::launch<Bf16>(map, p, stream) : lat::launch<F16>(map, p, stream);
}

}  // namespace mtpspec
