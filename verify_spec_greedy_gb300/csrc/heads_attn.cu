// Attention with grouped heads over the paged cache of keys and values.
//
// A CTA a (token, query head).  Each of its four warps takes every fourth visible key with the
// running maximum m and sum l of a softmax; a lane holds eight elements of the query, the key and
// the output.  The four warps' parts are joined at the end, each by 2^(m - m').
#include "common.cuh"
#include "half_types.cuh"
#include "kernels.h"

namespace mtpspec {
namespace hat {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr int WARPS = 4, THREADS = 32 * WARPS;

template <typename T>
__global__ void __launch_bounds__(THREADS) k_heads_attn(const HeadsAttnArgs a) {
    __shared__ int first_above, most_before;
    __shared__ float ms[WARPS], ls[WARPS], parts[WARPS][256];
    const int64_t t = blockIdx.x / a.Hq;
    const int h = static_cast<int>(blockIdx.x - t * a.Hq), g = h / (a.Hq / a.Hkv);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // ---- the token's row: the one before the first bound above the token
    const int Tq = static_cast<int>(a.Tq);
    const auto bound = [&](int i) { return min(max(a.cu_q[i], 0), Tq); };
    if (threadIdx.x == 0) {
        first_above = static_cast<int>(a.B) + 1;
        most_before = 0;
    }
    __syncthreads();
    bool bad = false;
    for (int i = threadIdx.x; i <= a.B; i += THREADS) {
        if (bound(i) > t) atomicMin(&first_above, i);
        bad |= a.cu_q[i] < 0 || a.cu_q[i] > Tq || (i > 0 && a.cu_q[i] < a.cu_q[i - 1]);
        if (i < a.B) bad |= a.kv_len[i] < 0 || a.kv_len[i] > a.max_pages * a.page_size;
    }
    if (bad && blockIdx.x == 0 && a.status) atomicOr(a.status, MTPSPEC_STATUS_BAD_PARAM);
    __syncthreads();
    const int b = first_above - 1;
    if (b < 0 || b >= a.B) return;  // outside every row
    for (int i = threadIdx.x; i <= b; i += THREADS) atomicMax(&most_before, bound(i));
    __syncthreads();
    const int q0 = most_before, nq = bound(b + 1) - q0;
    const int64_t most = a.max_pages * a.page_size, cap = (int64_t{1} << 31) - 256;
    const int len = static_cast<int>(min(static_cast<int64_t>(max(a.kv_len[b], 0)), most < cap ? most : cap));
    const int pos = len - nq + static_cast<int>(t - q0);
    const int64_t from = a.window > 0 ? static_cast<int64_t>(pos) - a.window + 1 : 0;  // the window's first
    const bool in = lane * 8 < a.D;
    float qf[8] = {}, acc[8] = {};
    if (in) half8_to_float<T>(*reinterpret_cast<const uint4 *>(a.q + t * a.q_tok + h * a.q_head + lane * 8), qf);
    const float scale2 = a.scale * LOG2E;
    float m = -INFINITY, l = 0.0f;
    for (int64_t j = warp; j <= pos; j += WARPS) {
        if (j >= a.sinks && j < from) {  // between the first tokens and the window
            j += (from - j) / WARPS * WARPS;
            if (j < from) j += WARPS;
            if (j > pos) break;
        }
        const int64_t page = j / a.page_size;
        const int id = a.block_table[b * a.max_pages + page];
        float kf[8] = {}, vf[8] = {};
        if (id >= 0 && id < a.num_pages) {
            if (in) {
                const int64_t at = id * a.page_stride + (j - page * a.page_size) * a.slot_stride +
                                   g * a.head_stride + lane * 8;
                half8_to_float<T>(*reinterpret_cast<const uint4 *>(a.k_cache + at), kf);
                half8_to_float<T>(*reinterpret_cast<const uint4 *>(a.v_cache + at), vf);
            }
        } else if (lane == 0 && a.status) {
            atomicOr(a.status, MTPSPEC_STATUS_BAD_PARAM);
        }
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) s += qf[k] * kf[k];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        s *= scale2;
        const float top = fmaxf(m, s);
        const float use = top == -INFINITY ? 0.0f : top;
        const float f = exp2f(m - use), p = exp2f(s - use);
        l = l * f + p;
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = acc[k] * f + p * vf[k];
        m = top;
    }
    if (lane == 0) {
        ms[warp] = m;
        ls[warp] = l;
    }
    if (in)
#pragma unroll
        for (int k = 0; k < 8; ++k) parts[warp][lane * 8 + k] = acc[k];
    __syncthreads();
    float top = -INFINITY, sum = 0.0f, w[WARPS];
    for (int i = 0; i < WARPS; ++i) top = fmaxf(top, ms[i]);
    const float use = top == -INFINITY ? 0.0f : top;
    for (int i = 0; i < WARPS; ++i) {
        w[i] = exp2f(ms[i] - use);
        sum += w[i] * ls[i];
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    for (int d = 2 * threadIdx.x; d < a.D; d += 2 * THREADS) {
        float x = 0.0f, y = 0.0f;
        for (int i = 0; i < WARPS; ++i) {
            x += w[i] * parts[i][d];
            y += w[i] * parts[i][d + 1];
        }
        *reinterpret_cast<uint32_t *>(a.out + t * a.out_tok + h * a.out_head + d) = T::narrow2(x * inv, y * inv);
    }
    if (threadIdx.x == 0 && a.lse)
        a.lse[t * a.Hq + h] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * LN2;
}

}  // namespace hat

size_t heads_attn_workspace_bytes(int64_t, int64_t, int32_t, int32_t, int32_t D) {
    return D <= 128 ? heads_chunk_workspace_bytes(D) : 256;
}

cudaError_t run_heads_attn(const HeadsAttnArgs &a, int dtype, cudaStream_t stream) {
    if (a.D <= 128) return run_heads_chunk(a, dtype, stream);
    const unsigned grid = static_cast<unsigned>(a.Tq * a.Hq);
    if (dtype == MTPSPEC_BF16)
        hat::k_heads_attn<Bf16><<<grid, hat::THREADS, 0, stream>>>(a);
    else
        hat::k_heads_attn<F16><<<grid, hat::THREADS, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace mtpspec
