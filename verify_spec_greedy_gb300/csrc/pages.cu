// The pages of a draft head's cache between two rounds of drafts: rows give pages back and take
// free ones, share those of another row, and live pages are moved together.  The description (a
// block table, the rows' counts, a reference count a page) stays on the device, and so do the
// pairs of pages that k_pages_copy then moves.
//
// Taking is a sequence by definition: the lowest free page to the first row that needs one.  In
// parallel it is two prefix sums, one of what the rows need and one of the free pages in order of
// their numbers, and the k-th page finds its row by a search in the first.  Both run in one CTA of
// 1024 threads, in windows of 8192 pages, until what is needed has been found: a barrier costs
// some 30 ns there, and a second launch or a grid-wide barrier some microseconds.
//
// The copy is bytes, 16 KB a step and CTA.
//
// Measured in a graph: resize of 256 rows, 40,000 pages of 16: 11 us, a chain of some ten loads and
// barriers and five windows (a call with 2^20 pages, of which the last are free: 320 us).  Fork of 64 rows
// into four, with the copy of their last pages, 67 MB: 21 us.  Compaction of 8192 pages with its copy, 93
// MB: 26 us, half of it the copy.
#include "common.cuh"
#include "kernels.h"

namespace mtpspec {
namespace pg {

constexpr int THREADS = 1024;
constexpr int WARPS = THREADS / 32;
constexpr int PER = 8;                 // pages of a window that a thread looks at
constexpr int WINDOW = THREADS * PER;
constexpr int LANES = 8;               // threads that give back a row's pages
constexpr unsigned ALL = 0xFFFFFFFFu;

__device__ __forceinline__ void flag(int32_t *status, int bit) {
    if (status) atomicOr(status, bit);
}

// The exclusive sum of every thread's value over the block, and the total.  `sums` is shared.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *sums, int64_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t at = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(ALL, at, o);
        if (lane >= o) at += x;
    }
    if (lane == 31) sums[warp] = at;
    __syncthreads();
    int64_t s = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(ALL, s, o);
        if (lane >= o) s += x;
    }
    total = __shfl_sync(ALL, s, 31);
    const int64_t before = __shfl_sync(ALL, s, warp == 0 ? 0 : warp - 1);
    __syncthreads();  // (the next sum may be written)
    return at - v + (warp == 0 ? 0 : before);
}

// The counts of a window's pages, as thread i looks at them: pages base + 1024 j + i, so that loads are
// whole lines.
struct Window {
    int32_t ref[PER];
    __device__ __forceinline__ void load(const int32_t *refs, int64_t base, int64_t end) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int64_t p = base + j * THREADS + threadIdx.x;
            ref[j] = p < end ? __ldcg(refs + p) : 0;
        }
    }
};
// Which pages of the window [base, base + WINDOW) a predicate holds for, in order of their numbers:
// calls put(rank in the window, page) for each, and returns how many there are.  `w` is the window,
// and then the one after it, on its way meanwhile.  `counts` is shared.
template <typename P, typename F>
__device__ __forceinline__ int window_ranks(const int32_t *refs, Window &w, int64_t base, int64_t end,
                                            int (*counts)[WARPS], const P &holds, const F &put) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned has[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int64_t p = base + j * THREADS + threadIdx.x;
        has[j] = __ballot_sync(ALL, p < end && holds(w.ref[j]));
        if (lane == 0) counts[j][warp] = __popc(has[j]);
    }
    w.load(refs, base + WINDOW, end);
    __syncthreads();
    // every warp adds up all counts, a column of eight a lane, and keeps its own places
    int total = 0, mine[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        int s = counts[j][lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(ALL, s, o);
            if (lane >= o) s += x;
        }
        const int before = __shfl_sync(ALL, s, warp == 0 ? 0 : warp - 1);
        mine[j] = total + (warp == 0 ? 0 : before);
        total += __shfl_sync(ALL, s, 31);
    }
#pragma unroll
    for (int j = 0; j < PER; ++j)
        if (has[j] >> lane & 1)
            put(mine[j] + __popc(has[j] & ((1u << lane) - 1)), base + j * THREADS + threadIdx.x);
    __syncthreads();  // (the next window's counts may be written)
    return total;
}

struct IsFree {
    __device__ bool operator()(int32_t r) const { return r == 0; }
};
struct IsLive {
    __device__ bool operator()(int32_t r) const { return r > 0; }
};

// What a row asks for.
struct Row {
    int held, kept;
    int64_t want;
    bool ok, partly;
};
__device__ __forceinline__ Row row_of(const PagesResizeArgs &a, int64_t b) {
    Row r;
    const int keep = a.keep[b], len = a.lens[b];
    r.held = a.held[b];
    const int64_t P = a.page_size;
    r.ok = keep >= 0 && r.held >= 0 && r.held <= a.max_pages && keep <= r.held * P && len >= keep &&
           len <= a.max_pages * P;
    r.kept = r.ok ? static_cast<int>((keep + P - 1) / P) : r.held;
    r.want = r.ok ? (len + P - 1) / P : r.held;
    r.partly = r.ok && keep % P != 0;
    return r;
}
// A writer of a shared page: a row whose last kept page is partly filled.  While rows agree on who
// stays, a page's count holds how many writers it has in its upper half; and when all its holders
// are writers, the lowest of them, as a negative number.
__device__ __forceinline__ int32_t code_of(const PagesResizeArgs &a, int64_t b) {
    return -static_cast<int32_t>(1 + a.B - b);
}
__device__ __forceinline__ bool is_page(const PagesResizeArgs &a, int32_t p) {
    return p >= 0 && p < a.num_pages;
}

__global__ void __launch_bounds__(THREADS) k_pages_resize(const PagesResizeArgs a) {
    __shared__ int64_t sums[WARPS], start[THREADS];
    __shared__ int counts[PER][WARPS];
    __shared__ unsigned leaving[16384 / 32];  // the rows that leave their last page
    const int tid = threadIdx.x;
    // (a thread's first row, which is its only one up to 1024 rows, stays in registers)
    Row mine = {};
    int32_t my_last = -1;
    if (tid < a.B) {
        mine = row_of(a, tid);
        if (mine.partly) my_last = a.block_table[tid * a.max_pages + mine.kept - 1];
    }
    const auto row = [&](int64_t b) { return b == tid ? mine : row_of(a, b); };
    const auto last_page = [&](int64_t b, const Row &r) {
        return b == tid ? my_last : r.partly ? a.block_table[b * a.max_pages + r.kept - 1] : -1;
    };
    // ---- 1. pages given back
    for (int64_t b = tid / LANES; b < a.B; b += THREADS / LANES) {
        const int keep = a.keep[b];
        const Row r = row_of(a, b);
        if (tid % LANES == 0 && !r.ok && keep >= 0) flag(a.status, MTPSPEC_STATUS_BAD_PARAM);
        int32_t *table = a.block_table + b * a.max_pages;
        for (int i = r.kept + tid % LANES; i < r.held && r.ok; i += LANES) {
            const int32_t p = table[i];
            table[i] = -1;
            if (is_page(a, p))
                atomicSub(a.refs + p, 1);
            else
                flag(a.status, MTPSPEC_STATUS_BAD_PARAM);
        }
    }
    for (int i = tid; i < 16384 / 32; i += THREADS) leaving[i] = 0;
    __syncthreads();
    // ---- 2. who leaves a page that others hold too
    bool shared = false;
    if (a.copies)
        for (int64_t b = tid; b < a.B; b += THREADS) {
            const Row r = row(b);
            const int32_t p = last_page(b, r);
            if (!is_page(a, p)) {
                if (r.partly) flag(a.status, MTPSPEC_STATUS_BAD_PARAM);
            } else if ((__ldcg(a.refs + p) & 0xFFFF) > 1) {
                atomicAdd(a.refs + p, 1 << 16);
                shared = true;
            }
        }
    if (__syncthreads_or(shared)) {
        for (int64_t b = tid; b < a.B; b += THREADS) {
            const int32_t p = last_page(b, row(b));
            if (!is_page(a, p)) continue;
            const int32_t v = __ldcg(a.refs + p);
            if (v < 0 || (v >> 16 > 0 && v >> 16 == (v & 0xFFFF))) atomicMin(a.refs + p, code_of(a, b));
        }
        __syncthreads();
        for (int64_t b = tid; b < a.B; b += THREADS) {
            const int32_t p = last_page(b, row(b));
            if (!is_page(a, p)) continue;
            const int32_t v = __ldcg(a.refs + p);
            if (v < 0 ? v != code_of(a, b) : v >> 16 > 0)
                atomicOr(&leaving[b >> 5], 1u << (b & 31));
        }
        __syncthreads();
        for (int64_t b = tid; b < a.B; b += THREADS) {  // the counts again, without those who leave
            const int32_t p = last_page(b, row(b));
            if (!is_page(a, p)) continue;
            const bool leaves = leaving[b >> 5] >> (b & 31) & 1;
            const int32_t v = __ldcg(a.refs + p);
            if (v == code_of(a, b))
                atomicExch(a.refs + p, 1);
            else if (v > 0 && leaves && v >> 16 > 0)
                atomicSub(a.refs + p, (1 << 16) + 1);
        }
        __syncthreads();
    }
    // ---- 3. what the rows need, a run of rows a thread
    Window window;
    window.load(a.refs, 0, a.num_pages);
    const int64_t run = (a.B + THREADS - 1) / THREADS, b0 = tid * run, b1 = min(b0 + run, a.B);
    const auto need_of = [&](int64_t b, const Row &r) {
        return max(r.want - r.kept, int64_t{0}) + (leaving[b >> 5] >> (b & 31) & 1);
    };
    int64_t need = 0, total;
    for (int64_t b = b0; b < b1; ++b) need += need_of(b, row(b));
    const int64_t at = block_scan(need, sums, total);
    start[tid] = at;
    __syncthreads();
    // ---- free pages, lowest first, each to the row that it falls to
    int64_t found = 0;
    for (int64_t base = 0; base < a.num_pages && found < total; base += WINDOW) {
        found += window_ranks(a.refs, window, base, a.num_pages, counts, IsFree{}, [&](int rank, int64_t page) {
            int64_t k = found + rank;
            if (k >= total) return;
            int lo = 0, hi = THREADS - 1;  // the last thread whose rows start at or before k
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (start[mid] <= k)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            k -= start[lo];
            for (int64_t b = lo * run;; ++b) {
                const Row r = row_of(a, b);
                const int64_t n = need_of(b, r);
                if (k >= n) {
                    k -= n;
                    continue;
                }
                const bool leaves = leaving[b >> 5] >> (b & 31) & 1;
                int32_t *table = a.block_table + b * a.max_pages + r.kept;
                if (leaves && k == 0) {
                    a.copies[2 * b] = table[-1];
                    a.copies[2 * b + 1] = static_cast<int32_t>(page);
                } else {
                    table[k - leaves] = static_cast<int32_t>(page);
                }
                a.refs[page] = 1;
                break;
            }
        });
    }
    __syncthreads();
    // ---- the rows' counts; a row that did not get all gives back what it got
    int64_t end = at;
    bool none = false;
    for (int64_t b = b0; b < b1; ++b) {
        const Row r = row(b);
        const int64_t n = need_of(b, r), first = end;
        end += n;
        const bool leaves = leaving[b >> 5] >> (b & 31) & 1;
        int32_t *table = a.block_table + b * a.max_pages;
        const bool got = end <= found;
        if (got) {
            if (leaves) table[r.kept - 1] = a.copies[2 * b + 1];
        } else if (n > 0) {
            none = true;
            for (int64_t k = 0; k < found - first; ++k) {
                int32_t *p = leaves && k == 0 ? a.copies + 2 * b + 1 : table + r.kept + k - leaves;
                a.refs[*p] = 0;
                *p = -1;
            }
            if (leaves) atomicAdd(a.refs + table[r.kept - 1], 1);
        }
        if (a.copies && !(leaves && got)) a.copies[2 * b] = a.copies[2 * b + 1] = -1;
        if (r.ok) a.held[b] = static_cast<int32_t>(got ? r.want : r.kept);
    }
    if (none) flag(a.status, MTPSPEC_STATUS_NO_PAGES);
}

// A CTA a pair of rows.
constexpr int FORK_THREADS = 256;

__global__ void __launch_bounds__(FORK_THREADS) k_pages_fork(const PagesForkArgs a) {
    const int i = blockIdx.x, src = a.src_rows[i], dst = a.dst_rows[i];
    bool bad = src < 0 || src >= a.B || dst < 0 || dst >= a.B;
    for (int j = threadIdx.x; j < a.n; j += FORK_THREADS) {
        const int d = a.dst_rows[j];
        bad |= d == src || (j > i && d == dst);
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) flag(a.status, MTPSPEC_STATUS_BAD_PARAM);
        return;
    }
    const int wide = static_cast<int>(a.max_pages);
    const int old = min(max(a.held[dst], 0), wide), now = min(max(a.held[src], 0), wide);
    const int32_t *from = a.block_table + src * a.max_pages;
    int32_t *to = a.block_table + dst * a.max_pages;
    bad = false;
    for (int e = threadIdx.x; e < max(old, now); e += FORK_THREADS) {
        const int32_t p = e < now ? from[e] : -1, q = e < old ? to[e] : -1;
        to[e] = p;
        if (p >= 0 && p < a.num_pages)
            atomicAdd(a.refs + p, 1);
        else
            bad |= e < now;
        if (q >= 0 && q < a.num_pages)
            atomicSub(a.refs + q, 1);
        else
            bad |= e < old;
    }
    if (bad) flag(a.status, MTPSPEC_STATUS_BAD_PARAM);
    __syncthreads();
    if (threadIdx.x == 0) a.held[dst] = now;
}

__global__ void __launch_bounds__(THREADS) k_pages_compact(const PagesCompactArgs a) {
    __shared__ int64_t sums[WARPS];
    __shared__ int counts[PER][WARPS];
    const IsLive live;
    Window window;
    int64_t mine = 0, L;
    for (int64_t base = 0; base < a.num_pages; base += WINDOW) {
        window.load(a.refs, base, a.num_pages);
#pragma unroll
        for (int j = 0; j < PER; ++j) mine += live(window.ref[j]);
    }
    block_scan(mine, sums, L);
    int n = 0, m = 0;
    window.load(a.refs, 0, L);
    for (int64_t base = 0; base < L; base += WINDOW)
        n += window_ranks(a.refs, window, base, L, counts, IsFree{}, [&](int rank, int64_t p) {
            a.moves[2 * (static_cast<int64_t>(n) + rank) + 1] = static_cast<int32_t>(p);
        });
    window.load(a.refs, L, a.num_pages);
    for (int64_t base = L; base < a.num_pages && m < n; base += WINDOW)
        m += window_ranks(a.refs, window, base, a.num_pages, counts, live, [&](int rank, int64_t p) {
            a.moves[2 * (static_cast<int64_t>(m) + rank)] = static_cast<int32_t>(p);
        });
    // (a negative count, which no row holds, is neither live nor free: then the two may differ)
    n = min(n, m);
    __syncthreads();
    for (int64_t i = threadIdx.x; i < a.num_pages / 2; i += THREADS) {
        int32_t *pair = a.moves + 2 * i;
        if (i < n) {
            const int32_t from = pair[0], to = pair[1];  // (put there by this block, behind a barrier)
            a.refs[to] = a.refs[from];
            a.refs[from] = 0;
        } else {
            pair[0] = pair[1] = -1;
        }
    }
    if (threadIdx.x == 0) *a.n_moves = n;
}

// The table's entries that have moved, by a search among the pairs.
constexpr int TABLE_THREADS = 256;

__global__ void __launch_bounds__(TABLE_THREADS) k_pages_table(const PagesCompactArgs a) {
    pdl_wait_primary();
    const int n = *a.n_moves;
    for (int64_t b = blockIdx.x; b < a.B; b += gridDim.x) {
        const int64_t held = min(static_cast<int64_t>(max(a.held[b], 0)), a.max_pages);
        int32_t *table = a.block_table + b * a.max_pages;
        for (int64_t e = threadIdx.x; e < held; e += TABLE_THREADS) {
            const int32_t p = table[e];
            if (p < 0 || p >= a.num_pages) {
                flag(a.status, MTPSPEC_STATUS_BAD_PARAM);
                continue;
            }
            int lo = 0, hi = n;  // the first pair from p on
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                if (a.moves[2 * static_cast<int64_t>(mid)] < p)
                    lo = mid + 1;
                else
                    hi = mid;
            }
            if (lo < n && a.moves[2 * static_cast<int64_t>(lo)] == p)
                table[e] = a.moves[2 * static_cast<int64_t>(lo) + 1];
        }
    }
}

constexpr int COPY_THREADS = 256;
constexpr int VPT = 4;                             // 16-byte vectors in flight a thread
constexpr int64_t STEP = COPY_THREADS * VPT;       // vectors a CTA moves at a time

__global__ void __launch_bounds__(COPY_THREADS)
k_pages_copy(const __grid_constant__ PagesCopyArgs a) {
    const int64_t n = a.n_pairs ? min(static_cast<int64_t>(max(*a.n_pairs, 0)), a.n) : a.n;
    const int64_t vecs = a.page_bytes / 16, steps = (vecs + STEP - 1) / STEP;
    const int64_t per = steps * a.n_caches, total = n * per;
    for (int64_t i = blockIdx.x; i < total; i += gridDim.x) {
        const int64_t pair = i / per, in = i - pair * per;
        const int c = static_cast<int>(in / steps);
        const int32_t from = a.pairs[2 * pair], to = a.pairs[2 * pair + 1];
        if (from < 0 || to < 0) continue;
        if (from >= a.num_pages || to >= a.num_pages) {
            if (threadIdx.x == 0) flag(a.status, MTPSPEC_STATUS_BAD_PARAM);
            continue;
        }
        const uint4 *src = reinterpret_cast<const uint4 *>(a.caches[c] + from * a.page_stride);
        uint4 *dst = reinterpret_cast<uint4 *>(a.caches[c] + to * a.page_stride);
        const int64_t first = (in - c * steps) * STEP + threadIdx.x;
        uint4 v[VPT];
#pragma unroll
        for (int u = 0; u < VPT; ++u)
            if (first + u * COPY_THREADS < vecs) v[u] = __ldcs(src + first + u * COPY_THREADS);
#pragma unroll
        for (int u = 0; u < VPT; ++u)
            if (first + u * COPY_THREADS < vecs) dst[first + u * COPY_THREADS] = v[u];
    }
}

}  // namespace pg

cudaError_t run_pages_resize(const PagesResizeArgs &a, cudaStream_t stream) {
    pg::k_pages_resize<<<1, pg::THREADS, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

cudaError_t run_pages_fork(const PagesForkArgs &a, cudaStream_t stream) {
    pg::k_pages_fork<<<static_cast<unsigned>(a.n), pg::FORK_THREADS, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

cudaError_t run_pages_compact(const PagesCompactArgs &a, cudaStream_t stream) {
    pg::k_pages_compact<<<1, pg::THREADS, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    count_launches(1);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.B < 2048 ? a.B : 2048));
    cfg.blockDim = dim3(pg::TABLE_THREADS);
    cfg.stream = stream;
    cfg.attrs = pdl_attr();
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, pg::k_pages_table, a);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

cudaError_t run_pages_copy(const PagesCopyArgs &a, cudaStream_t stream) {
    const int64_t steps = (a.page_bytes / 16 + pg::STEP - 1) / pg::STEP;
    const int64_t most = 152 * 8;  // all the CTAs that the GPU holds at a time
    const int64_t per = steps * a.n_caches;
    const int64_t total = a.n > most / per ? most : a.n * per;
    pg::k_pages_copy<<<static_cast<unsigned>(total < most ? total : most), pg::COPY_THREADS, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace mtpspec
