// What the kernels of the attention with grouped heads share: the units of work, their even cut
// over the CTAs, and the joining of the units that the cut divides.
#pragma once

#include "half_types.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace mtpspec {
namespace heads {

using namespace tg;

constexpr int SMS = 152;           // multiprocessors of a GB300
constexpr int64_t START = 3;       // a unit's start and end, in key tiles (in heads_chunk.cu 2: 5 % slower, 5: 1-7 %)
constexpr float LAZY = 8.0f;       // the running maximum may lag by a factor of 2^8
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr uint32_t POLL_LIMIT = 1u << 25;  // polls of some 20 ns: ~1 s

// For the joining kernel, by CTA: the unit that starts there and ends in another.
struct __align__(32) Plan {
    int q0, m0, rows, head, parts;  // its row's first token in q, its (token, head) rows, its key
                                    // head, the CTAs that have a part; 0 parts: there is none
};

struct Params {
    const int32_t *cu_q, *kv_len, *block_table;
    int64_t max_pages;
    int max_len;         // the table's positions, up to 2^31 - 256
    int num_pages, page_size, box_rows;
    int B, Tq, Hq, Hkv, G, D, window, sinks;
    int unit_rows;       // (token, head) rows that a unit holds
    float scale2;        // scale * log2(e), above 0
    const uint16_t *q;
    int64_t q_tok, q_head;
    uint16_t *out;
    int64_t out_tok, out_head;
    float *lse;
    Plan *plan;
    float *part;         // fp32, normalised partial outputs: two slots a CTA
    float *part_lse;     // base 2
    int32_t *status;
};

struct Maps {
    CUtensorMap q, k, v;
};

__device__ __forceinline__ int row_len(const Params &p, int b) {
    return min(max(p.kv_len[b], 0), p.max_len);
}
// Bound i of cu_q as it is taken: in [0, Tq], and not below the ones before it.
__device__ __forceinline__ int bound(const Params &p, int i, int before) {
    return max(min(p.cu_q[i], p.Tq), before);
}

// A unit of work: `unit_rows` (token, head) rows of one key head of a row, against tiles of TN keys.
// With a window it meets the tiles of the first tokens, then those of the window.
template <int TN>
struct Unit {
    int q0, nq, len, m0;  // the row's first token in q, its tokens and length; the unit's first row
    int w0, ns;           // the first key tile of its window, and the tiles of first tokens before
    __device__ __forceinline__ Unit() {}
    __device__ __forceinline__ Unit(const Params &p, int q0_, int nq_, int len_, int unit)
        : q0(q0_), nq(nq_), len(len_), m0(unit * p.unit_rows) {
        w0 = ns = 0;
        if (p.window > 0 && p.window < len) {
            w0 = window(p) / TN;
            ns = min(p.sinks / TN + (p.sinks % TN != 0), w0);
        }
    }
    // The first key of its first row's window: none of its rows sees one before it but the first tokens.
    __device__ __forceinline__ int window(const Params &p) const {
        return p.window > 0 && p.window < len ? max(0, len - nq + m0 / p.G - p.window + 1) : 0;
    }
    // Key tiles that `rows` rows from row m on meet.
    __device__ __forceinline__ int tiles(const Params &p, int m, int rows) const {
        const int hi = len - nq + min((m + rows - 1) / p.G + 1, nq);
        return m >= nq * p.G || hi <= 0 ? 0 : ns + (hi + TN - 1) / TN - w0;
    }
    __device__ __forceinline__ int tiles(const Params &p) const { return tiles(p, m0, p.unit_rows); }
    // Its length in the cut (one tile at least, so that every unit is somebody's).
    __device__ __forceinline__ int64_t weight(const Params &p) const { return START + max(tiles(p), 1); }
    // The number of its i-th key tile.
    __device__ __forceinline__ int key_tile(int i) const { return i < ns ? i : i - ns + w0; }
};

// An even cut of all units laid end to end: of the CTAs that take part, the first `rem` have
// per + 1, the others per.
struct Cut {
    int64_t total, per;
    int active, rem;
    __device__ __forceinline__ Cut(int64_t sum, int ctas) : total(sum) {
        active = static_cast<int>(sum < ctas ? sum : ctas);
        if (active == 0) {
            per = 0;
        } else if (sum < (int64_t{1} << 31)) {
            per = static_cast<uint32_t>(sum) / static_cast<uint32_t>(active);
        } else {
            per = sum / active;
        }
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

// A CTA's walk through its part of the cut, by one warp, all lanes alike.
template <int TN>
struct Walk {
    int row, q0, q1, len, head, unit, units;  // the next unit
    int64_t cur, at, end;                     // what is left of the CTA's part, and where the unit starts
    bool cut_here;                            // a unit starts here and ends in another CTA

    __device__ __forceinline__ void open_row(const Params &p) {
        q1 = bound(p, row + 1, q0);
        len = row_len(p, row);
        units = units_of(p, q1 - q0);
    }
    static __device__ __forceinline__ int units_of(const Params &p, int nq) {
        return (nq * p.G + p.unit_rows - 1) / p.unit_rows;
    }
    // The next unit with tiles for this CTA: tiles i0 .. i1 - 1 of n; false if there is none.
    __device__ __forceinline__ bool next(const Params &p, const Cut &cut, Unit<TN> &u, int &i0, int &i1, int &n) {
        while (cur < end) {
            while (unit >= units) {  // (rows without tokens have no units)
                unit = 0;
                if (units == 0 || ++head == p.Hkv) {
                    head = 0;
                    q0 = q1;
                    if (++row >= p.B) return false;
                    open_row(p);
                }
            }
            u = Unit<TN>(p, q0, q1 - q0, len, unit);
            n = max(u.tiles(p), 1);
            const int64_t base = at + START, s = max(cur, base), e = min(end, base + n);
            at = base + n;
            cur = min(end, at);
            ++unit;
            if (s >= e) continue;
            i0 = static_cast<int>(s - base);
            i1 = static_cast<int>(e - base);
            if (i0 == 0 && i1 < n && (threadIdx.x & 31) == 0) {
                cut_here = true;
                p.plan[blockIdx.x] = {q0, u.m0, min(p.unit_rows, (q1 - q0) * p.G - u.m0), head,
                                      cut.owner(base + n - 1) - static_cast<int>(blockIdx.x) + 1};
            }
            return true;
        }
        return false;
    }
    // A CTA without a cut unit says so.
    __device__ __forceinline__ void close(const Params &p) const {
        if ((threadIdx.x & 31) == 0 && !cut_here) p.plan[blockIdx.x] = {0, 0, 0, 0, 0};
    }
};

// The scan of the rows' units by a whole block of NT threads, a run of rows a thread, or, of few
// rows, a row a warp whose lanes share its units; then warp `who` sets its walk up.
struct Scan {
    int64_t sums[32];
    int64_t first_off;
    int first_row, first_q0;
};
template <int TN, int NT>
__device__ __forceinline__ Cut find_start(const Params &p, Scan &sh, int who, Walk<TN> &walk) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool wide = p.B <= NT / 32;
    const int run = wide ? 1 : (p.B + NT - 1) / NT;
    const int b0 = min(p.B, wide ? warp : static_cast<int>(threadIdx.x) * run), b1 = min(p.B, b0 + run);
    bool bad = false, order = false;
    int64_t sum = 0;
    const auto weigh = [&](int q0, int q1, int len, int from, int step) {
        int64_t w = 0;
        for (int i = from; i < Walk<TN>::units_of(p, q1 - q0); i += step)
            w += Unit<TN>(p, q0, q1 - q0, len, i).weight(p);
        return w;
    };
    for (int b = b0; b < b1; ++b) {
        const int c0 = p.cu_q[b], c1 = p.cu_q[b + 1], len = p.kv_len[b];
        order |= c0 < 0 || c1 > p.Tq || c1 < c0;
        bad |= len < 0 || len > p.max_len;
        if (!order) sum += weigh(c0, c1, min(max(len, 0), p.max_len), wide ? lane : 0, wide ? 32 : 1);
    }
    const bool disorder = __syncthreads_or(order);
    if (bad || order)
        if (blockIdx.x == 0 && p.status) atomicOr(p.status, MTPSPEC_STATUS_BAD_PARAM);
    int q_before = 0;  // the largest bound up to the first of the run, as taken
    if (disorder) {
        for (int b = 0; b < b0; ++b) q_before = bound(p, b, q_before);
        sum = 0;
        int q0 = b0 < b1 ? bound(p, b0, q_before) : 0;
        for (int b = b0; b < b1; ++b) {
            const int q1 = bound(p, b + 1, q0);
            sum += weigh(q0, q1, row_len(p, b), wide ? lane : 0, wide ? 32 : 1);
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
    for (int w = 0; w < NT / 32; ++w) {
        if (w == warp) at += total;
        total += sh.sums[w];
    }
    at -= sum;
    const Cut cut(total, gridDim.x);
    const int64_t t0 = cut.first(blockIdx.x), t1 = cut.first(blockIdx.x + 1);
    if (wide) {  // the row's sum is its whole warp's
        at = __shfl_sync(0xFFFFFFFFu, at, 0);
        sum = sh.sums[warp];
    }
    if (t0 < t1 && at <= t0 && t0 < at + sum && (!wide || lane == 0)) {
        int q0 = bound(p, b0, q_before), b = b0;
        int64_t off = t0 - at;
        for (; b + 1 < b1; ++b) {  // (a run of one row has nothing to look for)
            const int q1 = bound(p, b + 1, q0);
            const int64_t mine = weigh(q0, q1, row_len(p, b), 0, 1) * p.Hkv;
            if (off < mine) break;
            off -= mine;
            q0 = q1;
        }
        sh.first_row = b;
        sh.first_q0 = q0;
        sh.first_off = off;
    }
    __syncthreads();
    if (warp != who) return cut;
    walk.cur = walk.at = t0;
    walk.end = t1;
    walk.cut_here = false;
    if (t0 >= t1) return cut;
    walk.row = sh.first_row;
    walk.q0 = sh.first_q0;
    walk.open_row(p);
    // the row's units of one head, 32 at a time, until the one that t0 lies in
    int64_t off = sh.first_off, mine = weigh(walk.q0, walk.q1, walk.len, lane, 32);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, o);
    walk.head = static_cast<int>(off / mine);
    off -= walk.head * mine;
    for (walk.unit = 0;; walk.unit += 32) {
        const int i = walk.unit + lane;
        const int64_t w = i < walk.units ? Unit<TN>(p, walk.q0, walk.q1 - walk.q0, walk.len, i).weight(p) : 0;
        int64_t to = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xFFFFFFFFu, to, o);
            if (lane >= o) to += v;
        }
        const int64_t here = __shfl_sync(0xFFFFFFFFu, to, 31);
        if (off < here || walk.unit + 32 >= walk.units) {
            const unsigned has = __ballot_sync(0xFFFFFFFFu, off < to);
            const int src = has ? __ffs(has) - 1 : 0;
            off -= __shfl_sync(0xFFFFFFFFu, to - w, src);
            walk.unit += src;
            break;
        }
        off -= here;
    }
    walk.at = t0 - off;
    return cut;
}

// A bounded wait; once any wait of the CTA has given up, the others return at once, and the roles run
// to their ends without touching what they could not wait for.
template <typename Shared>
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
template <typename Shared>
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
template <typename Shared>
__device__ __forceinline__ bool wait_far(Shared &sh, uint64_t *bar, uint32_t parity) {
    return wait_long(sh, bar, parity, 64 * WAIT_LIMIT);
}
// The bounded wait of a CTA that leaves, whatever the abort flag says.
__device__ __forceinline__ void wait_out(uint64_t *bar, uint32_t parity) {
    for (uint32_t it = 0; it < WAIT_LIMIT; ++it)
        if (mbar_test(bar, parity)) return;
}

// A tile of keys in boxes that stay within a page, one a lane: where this lane's box of the tile lies.
// Its page's number is asked for by look() and looked at by settle(), a tile later, so that nothing
// waits for the answer.  Of a box between the first tokens and the window, which no row of the unit
// sees, neither the table's entry nor the page is read: the entry may be gone, and the page another's.
struct Box {
    int page, slot;
    bool mine;
    __device__ __forceinline__ void look(const Params &p, const int32_t *table, int key, int len, int window,
                                         bool lane_has) {
        const int pi = key / p.page_size;
        slot = key - pi * p.page_size;
        mine = lane_has && key < len && (key + p.box_rows > window || key < p.sinks);
        if (mine) page = table[pi];
    }
    // (page, row of it): where nothing is seen, and where the table has no such page, TMA fills zeros
    __device__ __forceinline__ int2 settle(const Params &p) const {
        const bool good = mine && static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages);
        if (mine && !good && p.status) atomicOr(p.status, MTPSPEC_STATUS_BAD_PARAM);
        return make_int2(good ? page : p.num_pages, slot);
    }
};

// Partial outputs lie by fours of columns, the rows side by side (a thread that has a row's columns
// writes beside its neighbours): float4 number (slot * 16 NC + column / 4) * TM + row.
template <int NC, int TM>
__device__ __forceinline__ float4 *part_at(const Params &p, int slot, int column, int row) {
    return reinterpret_cast<float4 *>(p.part) +
           (static_cast<int64_t>(slot) * (16 * NC) + column / 4) * TM + row;
}

// Units cut among CTAs: each row's partial outputs, weighted by their sums, become the output.  A
// block takes 32 rows, a row a lane; blockIdx.y is the CTA of the first kernel in which the unit
// starts.  Its eight warps take the columns, or, with SPREAD, for units cut into many parts, an
// eighth of the parts each, and blockIdx.z the columns.
constexpr int JOIN_THREADS = 256, JOIN_WARPS = JOIN_THREADS / 32;

template <typename T, int NC, int TM, bool SPREAD>
__global__ void __launch_bounds__(JOIN_THREADS) k_heads_join(const Params p) {
    constexpr int COLS = 8 * NC, QUADS = 2 * NC;  // of a warp
    __shared__ float shared[SPREAD ? JOIN_WARPS : 1][SPREAD ? 32 : 1][COLS + 2];
    pdl_wait_primary();
    const Plan u = p.plan[blockIdx.y];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.x * 32 + lane;
    // (what an aborted call left there is checked)
    if (u.parts < 2 || u.parts > static_cast<int>(gridDim.y - blockIdx.y) || u.q0 < 0 || u.m0 < 0 ||
        u.q0 + (u.m0 + u.rows - 1) / p.G >= p.Tq || u.head < 0 || u.head >= p.Hkv ||
        static_cast<int>(blockIdx.x) * 32 >= u.rows)
        return;
    // a CTA's partial: the second slot where the unit starts, else the first
    const auto slot = [&](int i) { return static_cast<int>(2 * (blockIdx.y + i) + (i == 0)); };
    const auto lse2 = [&](int i) { return p.part_lse[static_cast<int64_t>(slot(i)) * TM + r]; };
    const bool real = r < u.rows;
    const int col = (SPREAD ? blockIdx.z : warp) * COLS;
    float top = -INFINITY, sum = 0.0f;
    float acc[COLS] = {};
    if (real) {
#pragma unroll 4
        for (int i = 0; i < u.parts; ++i) top = fmaxf(top, lse2(i));
        const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll 4
        for (int i = SPREAD ? warp : 0; i < u.parts; i += SPREAD ? JOIN_WARPS : 1) {
            const float w = exp2f(lse2(i) - ref);
            float4 v[QUADS];
#pragma unroll
            for (int k = 0; k < QUADS; ++k) v[k] = *part_at<NC, TM>(p, slot(i), col + 4 * k, r);
            sum += w;
#pragma unroll
            for (int k = 0; k < QUADS; ++k) {
                acc[4 * k] += w * v[k].x;
                acc[4 * k + 1] += w * v[k].y;
                acc[4 * k + 2] += w * v[k].z;
                acc[4 * k + 3] += w * v[k].w;
            }
        }
    }
    if (SPREAD) {
#pragma unroll
        for (int k = 0; k < COLS; ++k) shared[warp][lane][k] = acc[k];
        shared[warp][lane][COLS] = sum;
        __syncthreads();
        if (warp != 0) return;
#pragma unroll
        for (int w = 1; w < JOIN_WARPS; ++w) {
#pragma unroll
            for (int k = 0; k < COLS; ++k) acc[k] += shared[w][lane][k];
            sum += shared[w][lane][COLS];
        }
    }
    if (!real) return;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int m = u.m0 + r, tok = m / p.G, head = u.head * p.G + m - tok * p.G;
    const int64_t out_row = u.q0 + tok;
    uint16_t *dst = p.out + out_row * p.out_tok + head * p.out_head + col;
#pragma unroll
    for (int k = 0; k < COLS; k += 8) {
        if (col + k >= p.D) break;
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = acc[k + i] * inv;
        *reinterpret_cast<uint4 *>(dst + k) = float_to_half8<T>(f);
    }
    if (p.lse && col == 0) p.lse[out_row * p.Hq + head] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * LN2;
}

// The joining kernel behind one that was launched with `cfg`.
template <typename T, int NC, int TM>
cudaError_t launch_join(cudaLaunchConfig_t cfg, const Params &p, cudaStream_t stream) {
    const unsigned ctas = cfg.gridDim.x;
    // very few units are cut into very many parts each (where they are eight in 19 parts, either way takes
    // the same; five parts are slower when spread, by 1.5 us)
    const int64_t units = static_cast<int64_t>(p.B) * p.Hkv + static_cast<int64_t>(p.Tq) * p.Hq / p.unit_rows;
    const bool spread = units * 32 < static_cast<int64_t>(ctas);
    cfg.gridDim = dim3(TM / 32, ctas, spread ? JOIN_WARPS : 1);
    cfg.blockDim = dim3(JOIN_THREADS);
    cfg.dynamicSmemBytes = 0;
    cfg.stream = stream;
    const cudaError_t e = spread ? cudaLaunchKernelEx(&cfg, k_heads_join<T, NC, TM, true>, p)
                                 : cudaLaunchKernelEx(&cfg, k_heads_join<T, NC, TM, false>, p);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

// The parameters and tensor maps of a call whose units hold `unit_rows` rows; the workspace's parts lie
// at the given offsets.  The queries' map, if it is asked for, brings a unit's, as unit_rows / G tokens
// of G heads.
inline bool set_up(const HeadsAttnArgs &a, int unit_rows, int TN, bool q_map, size_t plan,
                   size_t part, size_t lse, Params &p, Maps &maps) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    p = {};
    p.G = a.Hq / a.Hkv;
    p.unit_rows = unit_rows;
    // boxes of the largest power of two (up to a tile) that divides the page: a box never leaves
    // its page, and its rows start at a multiple of eight, the swizzle's period
    const int two = a.page_size & -a.page_size;
    p.box_rows = two < TN ? two : TN;
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
    const cuuint64_t cd[4] = {u(a.D), u(a.page_size), u(a.Hkv), u(a.num_pages)},
                     cs[3] = {u(slot * 2), u(head * 2), u(page * 2)};
    const cuuint32_t cb[4] = {64, static_cast<cuuint32_t>(p.box_rows), 1, 1};
    if (!encode(&maps.k, a.k_cache, cd, cs, cb) || !encode(&maps.v, a.v_cache, cd, cs, cb)) return false;
    if (q_map) {
        const cuuint64_t qd[4] = {u(a.D), u(p.G), u(a.Tq), u(a.Hkv)},
                         qs[3] = {u(q_head * 2), u(q_tok * 2), u(q_head * p.G * 2)};
        const cuuint32_t qb[4] = {64, static_cast<cuuint32_t>(p.G), static_cast<cuuint32_t>(unit_rows / p.G), 1};
        if (!encode(&maps.q, a.q, qd, qs, qb)) return false;
    } else {
        maps.q = maps.k;
    }
    unsigned char *ws = static_cast<unsigned char *>(a.workspace);
    p.cu_q = a.cu_q;
    p.kv_len = a.kv_len;
    p.block_table = a.block_table;
    p.max_pages = a.max_pages;
    const int64_t slots = a.max_pages * a.page_size, most = (int64_t{1} << 31) - 256;
    p.max_len = static_cast<int>(slots < most ? slots : most);
    p.num_pages = static_cast<int>(a.num_pages);
    p.page_size = a.page_size;
    p.B = static_cast<int>(a.B);
    p.Tq = static_cast<int>(a.Tq);
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.D = a.D;
    p.window = a.window;
    p.sinks = a.sinks;
    p.scale2 = a.scale * LOG2E;
    p.q = a.q;
    p.q_tok = a.q_tok;
    p.q_head = a.q_head;
    p.out = a.out;
    p.out_tok = a.out_tok;
    p.out_head = a.out_head;
    p.lse = a.lse;
    p.plan = reinterpret_cast<Plan *>(ws + plan);
    p.part = reinterpret_cast<float *>(ws + part);
    p.part_lse = reinterpret_cast<float *>(ws + lse);
    p.status = a.status;
    return true;
}

}  // namespace heads
}  // namespace mtpspec
