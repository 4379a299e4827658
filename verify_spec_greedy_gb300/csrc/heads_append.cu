// The append to the paged cache of keys and values: the heads' norms, the rotation of a part of
// each head, and the stores to the tokens' slots, in one launch.
//
// The work is bytes: every value is read once and written once; a norm is two operations an
// element, a rotation three.  A head of D elements lies in D / 8 lanes, 16 bytes a lane, so that
// a warp holds 1 to 16 heads at a time (two at D = 128) and a head's sum of squares is a few
// shuffles; the rotation's partner is in the same lane (neighbouring pairs) or R / 16 lanes on
// (pairs of the two halves: eight shuffles).  All heads of a token, queries, keys and values, are
// one list that warps take in runs, so the angles and the weights are loaded once a run.
//
// What bounds it (in a graph): 11,994 tokens, 16 / 4 heads of 256 of which 64 elements are turned, 298 MB:
// 73 us, 4.1 TB/s, 0.60 of the copy rate.  The issue slots are 76 % taken, by conversions, sums and
// addresses; loads ahead through registers or shared memory made it slower (84 and 104 us), runs of
// eight groups the same, of two 91 us.  1024 tokens, 32 / 8 heads of 128: 10.8 us.  One token: 2.7 us, the
// launch.
#include "common.cuh"
#include "half_types.cuh"
#include "kernels.h"

namespace mtpspec {
namespace hap {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;

// A run of U groups of heads of token t, whose values x are on their way.
template <typename T, bool PAIRS, int U>
__device__ __forceinline__ void append_run(const HeadsAppendArgs &a, const uint4 (&x)[U], const int (&h)[U],
                                           int64_t t, int run, int row, int pos, int lpv, int vec, bool in, int nq) {
    const int lane = threadIdx.x & 31, per = 32 / lpv;
    const bool good = row >= 0 && row < a.B && pos >= 0 && pos < a.pos_end;
    int page = -1, off = 0;
    if (good) {
        const int pi = pos / a.page_size;
        off = pos - pi * a.page_size;
        page = a.block_table[static_cast<int64_t>(row) * a.max_pages + pi];
        if (page >= a.num_pages) page = -1;
    }
    if (run == 0 && lane == 0 && a.status && row >= 0 && (!good || page < 0))
        atomicOr(a.status, MTPSPEC_STATUS_BAD_PARAM);
    if (!good) return;
    // this lane's angles, its partner, and the weights of its elements
    const bool turned = vec * 8 < a.R;
    float c[8], s[8];
    int from = lane;
    bool second = false;
    if (turned) {
        const float *angles = a.cos_sin + static_cast<int64_t>(pos) * a.R;
        if (PAIRS) {
            *reinterpret_cast<float4 *>(c) = *reinterpret_cast<const float4 *>(angles + 4 * vec);
            *reinterpret_cast<float4 *>(s) = *reinterpret_cast<const float4 *>(angles + a.R / 2 + 4 * vec);
        } else {
            const int half = a.R / 16;
            second = vec >= half;
            from = second ? lane - half : lane + half;
            const int i0 = 8 * (second ? vec - half : vec);
#pragma unroll
            for (int k = 0; k < 8; k += 4) {
                *reinterpret_cast<float4 *>(c + k) = *reinterpret_cast<const float4 *>(angles + i0 + k);
                *reinterpret_cast<float4 *>(s + k) = *reinterpret_cast<const float4 *>(angles + a.R / 2 + i0 + k);
            }
        }
    }
    uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
    if (in && a.q_norm_w && run * U * per < nq) wq = *reinterpret_cast<const uint4 *>(a.q_norm_w + vec * 8);
    if (in && a.k_norm_w) wk = *reinterpret_cast<const uint4 *>(a.k_norm_w + vec * 8);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int g = h[u] - nq;
        const bool query = g < 0, value = g >= a.Hkv;
        if (__all_sync(0xFFFFFFFFu, value || h[u] < 0)) {  // a group of values: as they are
            if (h[u] >= 0 && page >= 0)
                *reinterpret_cast<uint4 *>(a.v_cache + page * a.page_stride + off * a.slot_stride +
                                           (g - a.Hkv) * a.head_stride + vec * 8) = x[u];
            continue;
        }
        float f[8];
        half8_to_float<T>(x[u], f);
        // (all lanes take part in the shuffles, whatever they hold)
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += f[k] * f[k];
        for (int o = lpv >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (!value && (query ? a.q_norm_w : a.k_norm_w)) {
            const float inv = rsqrtf(sum / static_cast<float>(a.D) + a.eps);
            float w[8];
            half8_to_float<T>(query ? wq : wk, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = f[k] * inv * w[k];
        }
        float y[8];
        if (PAIRS) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                y[2 * k] = f[2 * k] * c[k] - f[2 * k + 1] * s[k];
                y[2 * k + 1] = f[2 * k] * s[k] + f[2 * k + 1] * c[k];
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float other = __shfl_sync(0xFFFFFFFFu, f[k], from);
                y[k] = second ? other * s[k] + f[k] * c[k] : f[k] * c[k] - other * s[k];
            }
        }
        if (h[u] < 0) continue;
        const uint4 out = value ? x[u] : float_to_half8<T>(turned ? y : f);
        if (query) {
            *reinterpret_cast<uint4 *>(a.q_out + t * a.q_out_tok + h[u] * a.q_out_head + vec * 8) = out;
        } else if (page >= 0) {
            uint16_t *cache = value ? a.v_cache : a.k_cache;
            *reinterpret_cast<uint4 *>(cache + page * a.page_stride + off * a.slot_stride +
                                       (value ? g - a.Hkv : g) * a.head_stride + vec * 8) = out;
        }
    }
}

// A warp a run of U groups.
template <typename T, bool PAIRS, int U>
__global__ void __launch_bounds__(THREADS, U <= 4 ? 4 : 3)
k_heads_append(const HeadsAppendArgs a, const uint32_t lpv, const uint32_t heads, const uint32_t runs) {
    const uint32_t lane = threadIdx.x & 31, warp = blockIdx.x * WARPS + (threadIdx.x >> 5);
    const uint32_t tok = warp / runs, run = warp - tok * runs;  // (at most 2^20 tokens x 768 runs)
    const int64_t t = tok;
    if (t >= a.T) return;
    const int per = 32 / lpv, sub = lane / lpv, vec = lane - sub * lpv;
    const bool in = vec * 8 < a.D;
    const int nq = a.q ? a.Hq : 0;
    // the values are loaded before the token's position is known: the two chains overlap
    uint4 x[U];
    int h[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        h[u] = (run * U + u) * per + sub;
        x[u] = make_uint4(0, 0, 0, 0);
        if (!in || h[u] >= static_cast<int>(heads)) {
            h[u] = -1;
            continue;
        }
        const int g = h[u] - nq;
        const uint16_t *src = g < 0          ? a.q + t * a.q_tok + h[u] * a.q_head
                              : g < a.Hkv ? a.k + t * a.k_tok + g * a.k_head
                                          : a.v + t * a.v_tok + (g - a.Hkv) * a.v_head;
        x[u] = *reinterpret_cast<const uint4 *>(src + vec * 8);
    }
    append_run<T, PAIRS, U>(a, x, h, t, run, a.tok_row[t], a.positions[t], lpv, vec, in, nq);
}

template <typename T, int U>
cudaError_t launch(const HeadsAppendArgs &a, int lpv, int heads, cudaStream_t stream) {
    const int run = U * (32 / lpv), runs = (heads + run - 1) / run;
    const unsigned grid = static_cast<unsigned>((a.T * runs + WARPS - 1) / WARPS);
    if (a.interleaved)
        k_heads_append<T, true, U><<<grid, THREADS, 0, stream>>>(a, lpv, heads, runs);
    else
        k_heads_append<T, false, U><<<grid, THREADS, 0, stream>>>(a, lpv, heads, runs);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}
template <typename T>
cudaError_t pick(const HeadsAppendArgs &a, cudaStream_t s) {
    int lpv = 2;
    while (lpv * 8 < a.D) lpv *= 2;
    const int heads = (a.q ? a.Hq : 0) + 2 * a.Hkv;
    // few heads in all are spread over as many warps as there are, many keep four groups a warp in
    // flight
    const int64_t groups = (static_cast<int64_t>(heads) * lpv + 31) / 32 * a.T;
    return groups >= 4 * 152 * 24 ? launch<T, 4>(a, lpv, heads, s) : launch<T, 1>(a, lpv, heads, s);
}

}  // namespace hap

cudaError_t run_heads_append(const HeadsAppendArgs &a, int dtype, cudaStream_t stream) {
    return dtype == MTPSPEC_BF16 ? hap::pick<Bf16>(a, stream) : hap::pick<F16>(a, stream);
}

}  // namespace mtpspec
