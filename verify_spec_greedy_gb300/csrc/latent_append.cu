// The paged latent cache's append: each token's latent (RMS-normalised when a weight is
// given) and its rotated key part go to the token's slot, and the heads' query parts are
// rotated by the same angles, in one launch.
//
// The work is bytes: every value is read once and written once, and a rotation is four
// products a pair.  Two kinds of CTA share the grid.  The first blocks take the queries, in
// units of 16 elements (two 16-byte loads and stores): eight neighbouring pairs, or eight pairs
// of the two halves, so that a unit's cosines and sines are two runs of 32 bytes either way.
// The blocks behind them take a token a warp: the latent stays in registers between the sum of
// squares and the scaling (at most 512 values, two vectors a lane).
//
// Few calls are long enough to be bound by HBM: the bound is the chain position - angles -
// stores of a block times the blocks that an SM goes through, so a thread loads two units
// before it needs their positions.  12k tokens x 32 heads (126 MB, in a graph): 24.5 us, 5.1
// TB/s, against 28.6 with one unit a thread and 27.5 with four (80 registers, fewer threads);
// 1024 tokens x 128 heads: 8.9 us against 9.4 and 9.5; from 4 to 64 tokens the same or better.
// One token: 3.1 us, the launch.
#include "common.cuh"
#include "kernels.h"
#include "half_types.cuh"

namespace mtpspec {
namespace la {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int UNITS = 2;  // units of sixteen query elements a thread takes, THREADS apart

// Where a token's row goes: `angle` says whether its row and position are good, `page`
// is its page or -1 (a padding token, or one that is not written).
struct Slot {
    bool angle, bad;
    int pos;
    int64_t page;
    int off;
};

__device__ __forceinline__ Slot find_slot(const LatentAppendArgs &a, int64_t t) {
    Slot s;
    const int row = a.tok_row[t];
    s.pos = a.positions[t];
    s.page = -1;
    s.off = 0;
    s.bad = false;
    s.angle = row >= 0 && row < a.B && s.pos >= 0 && s.pos < a.pos_end;
    if (row < 0) return s;
    if (!s.angle) {
        s.bad = true;
        return s;
    }
    const int pi = s.pos / a.page_size;
    const int page = a.block_table[static_cast<int64_t>(row) * a.max_pages + pi];
    if (page < 0 || page >= a.num_pages) {
        s.bad = true;
        return s;
    }
    s.page = page;
    s.off = s.pos - pi * a.page_size;
    return s;
}

// Sixteen elements of one vector of R values, the pairs i0 .. i0 + 7.
struct Sixteen {
    uint4 lo, hi;
};
template <bool PAIRS>
__device__ __forceinline__ int lo_of(int i0) { return PAIRS ? 2 * i0 : i0; }
template <bool PAIRS>
__device__ __forceinline__ int hi_of(int i0, int R) { return PAIRS ? 2 * i0 + 8 : R / 2 + i0; }
template <bool PAIRS>
__device__ __forceinline__ Sixteen load16(const uint16_t *x, int R, int i0) {
    return {*reinterpret_cast<const uint4 *>(x + lo_of<PAIRS>(i0)),
            *reinterpret_cast<const uint4 *>(x + hi_of<PAIRS>(i0, R))};
}
template <typename T, bool PAIRS>
__device__ __forceinline__ void rotate16(const Sixteen &x, uint16_t *y, const float *__restrict__ angles,
                                         int R, int i0) {
    float c[8], s[8], a[8], b[8];
#pragma unroll
    for (int u = 0; u < 8; u += 4) {
        *reinterpret_cast<float4 *>(c + u) = *reinterpret_cast<const float4 *>(angles + i0 + u);
        *reinterpret_cast<float4 *>(s + u) = *reinterpret_cast<const float4 *>(angles + R / 2 + i0 + u);
    }
    half8_to_float<T>(x.lo, a);
    half8_to_float<T>(x.hi, b);
    float o0[8], o1[8];
    if (PAIRS) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            o0[2 * u] = a[2 * u] * c[u] - a[2 * u + 1] * s[u];
            o0[2 * u + 1] = a[2 * u] * s[u] + a[2 * u + 1] * c[u];
            o1[2 * u] = b[2 * u] * c[4 + u] - b[2 * u + 1] * s[4 + u];
            o1[2 * u + 1] = b[2 * u] * s[4 + u] + b[2 * u + 1] * c[4 + u];
        }
    } else {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            o0[u] = a[u] * c[u] - b[u] * s[u];
            o1[u] = a[u] * s[u] + b[u] * c[u];
        }
    }
    *reinterpret_cast<uint4 *>(y + lo_of<PAIRS>(i0)) = float_to_half8<T>(o0);
    *reinterpret_cast<uint4 *>(y + hi_of<PAIRS>(i0, R)) = float_to_half8<T>(o1);
}

template <typename T, bool PAIRS>
__global__ void __launch_bounds__(THREADS)
k_append(const LatentAppendArgs a, const unsigned q_blocks) {
    const uint32_t units = a.R / 16;  // units of 16 elements in one vector of R
    if (blockIdx.x < q_blocks) {
        // (at most 2^20 tokens x 1024 heads x 4 units: the last index is 2^32 - 1)
        const uint32_t per_tok = static_cast<uint32_t>(a.Hq) * units;
        const uint32_t first = blockIdx.x * (THREADS * UNITS) + threadIdx.x;
        // the values are loaded before the token's position is known: the two chains overlap
        Sixteen x[UNITS];
        int pos[UNITS];
        uint16_t *y[UNITS];
        uint32_t i0[UNITS];
#pragma unroll
        for (int k = 0; k < UNITS; ++k) {
            const uint32_t i = first + k * THREADS, t = i / per_tok;
            pos[k] = -1;
            if (t >= a.T) continue;
            const uint32_t r = i - t * per_tok, h = r / units;
            i0[k] = 8 * (r - h * units);
            x[k] = load16<PAIRS>(a.q_rot + t * a.q_rot_tok + h * a.q_rot_head, a.R, i0[k]);
            y[k] = a.q_out + t * a.q_out_tok + h * a.q_out_head;
            const int row = a.tok_row[t];
            pos[k] = a.positions[t];
            if (row < 0 || row >= a.B || pos[k] >= a.pos_end) pos[k] = -1;
        }
#pragma unroll
        for (int k = 0; k < UNITS; ++k)
            if (pos[k] >= 0)
                rotate16<T, PAIRS>(x[k], y[k], a.cos_sin + static_cast<int64_t>(pos[k]) * a.R, a.R, i0[k]);
        return;
    }
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x - q_blocks) * WARPS + (threadIdx.x >> 5);
    if (t >= a.T) return;
    // the token's own values are loaded before its slot is known: the two chains overlap
    const int vecs = a.L / 8;
    const uint16_t *x = a.latent + t * a.latent_stride;
    uint4 v[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (lane + 32 * k < vecs) v[k] = ld_stream_16B(x + 8 * (lane + 32 * k));
    Sixteen rot;
    if (lane < units) rot = load16<PAIRS>(a.rot + t * a.rot_stride, a.R, 8 * lane);
    const Slot s = find_slot(a, t);
    if (s.bad && lane == 0 && a.status) atomicOr(a.status, MTPSPEC_STATUS_BAD_PARAM);
    if (s.page < 0) return;
    uint16_t *dst = a.cache + s.page * a.page_stride + static_cast<int64_t>(s.off) * (a.L + a.R);
    if (lane < units)
        rotate16<T, PAIRS>(rot, dst + a.L,
                           a.cos_sin + static_cast<int64_t>(s.pos) * a.R, a.R, 8 * lane);
    if (a.norm_w) {
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (lane + 32 * k < vecs) {
                float f[8];
                half8_to_float<T>(v[k], f);
#pragma unroll
                for (int u = 0; u < 8; ++u) sum += f[u] * f[u];
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        const float inv = rsqrtf(sum / static_cast<float>(a.L) + a.eps);
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (lane + 32 * k < vecs) {
                float f[8], w[8];
                half8_to_float<T>(v[k], f);
                half8_to_float<T>(*reinterpret_cast<const uint4 *>(a.norm_w + 8 * (lane + 32 * k)), w);
#pragma unroll
                for (int u = 0; u < 8; ++u) f[u] = f[u] * inv * w[u];
                v[k] = float_to_half8<T>(f);
            }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (lane + 32 * k < vecs) *reinterpret_cast<uint4 *>(dst + 8 * (lane + 32 * k)) = v[k];
}

template <typename T, bool PAIRS>
cudaError_t launch(const LatentAppendArgs &a, cudaStream_t stream) {
    const int64_t q_units = a.q_rot ? a.T * a.Hq * (a.R / 16) : 0;
    const int64_t a_block = int64_t{THREADS} * UNITS;
    const unsigned q_blocks = static_cast<unsigned>((q_units + a_block - 1) / a_block);
    const unsigned t_blocks = static_cast<unsigned>((a.T + WARPS - 1) / WARPS);
    k_append<T, PAIRS><<<q_blocks + t_blocks, THREADS, 0, stream>>>(a, q_blocks);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace la

cudaError_t run_latent_append(const LatentAppendArgs &a, int dtype, cudaStream_t stream) {
    if (dtype == MTPSPEC_BF16)
        return a.interleaved ? la::launch<Bf16, true>(a, stream) : la::launch<Bf16, false>(a, stream);
    return a.interleaved ? la::launch<F16, true>(a, stream) : la::launch<F16, false>(a, stream);
}

}  // namespace mtpspec
