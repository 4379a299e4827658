// The 16-bit element types of the latent attention, as tags, and their conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace mtpspec {

struct Bf16 {
    static constexpr uint32_t mma_format = 1;  // operand format field of kind::f16
    // A softmax's first weight, in powers of two, when it is rounded to this type: bf16 has the
    // exponents of fp32, and its smallest weights are worth as many bits as the largest.
    static constexpr float first_weight = 0.0f;
    static __device__ __forceinline__ float2 widen2(uint32_t v) {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t narrow2(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};

struct F16 {
    static constexpr uint32_t mma_format = 0;
    // fp16's normal values end at 2^-14 and its largest is just below 2^16.  Weights start at 2^7
    // and, while the maximum they refer to lags by up to 2^8, stay within 2^15; so those down to
    // 2^-21 of the first keep all their bits, those down to 2^-32 some.  (From 1, keys 2^-18 below
    // an early high one were off by up to 2^-7: a fair part of the output when they are many.)
    static constexpr float first_weight = 7.0f;
    static __device__ __forceinline__ float2 widen2(uint32_t v) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&v));
    }
    static __device__ __forceinline__ uint32_t narrow2(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};

template <typename T>
__device__ __forceinline__ void half8_to_float(const uint4 &v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = T::widen2(w[i]);
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
    }
}
template <typename T>
__device__ __forceinline__ uint4 float_to_half8(const float (&f)[8]) {
    return make_uint4(T::narrow2(f[0], f[1]), T::narrow2(f[2], f[3]), T::narrow2(f[4], f[5]),
                      T::narrow2(f[6], f[7]));
}

}  // namespace mtpspec
