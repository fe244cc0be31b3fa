// mx_block.cuh -- the MXFP8 / MXFP4 quantizer of one block of 32 bf16 values
// (sm_100a), shared by the tensor quantizer (mx.cu, which states the method) and
// the cache writer (cache.cu).
#pragma once

#include "mxq_device.cuh"
#include "mxq.h"

namespace mxq {

template <int FMT>
__device__ __forceinline__ int mx_exponent(uint32_t amax_bits)
{
    constexpr int k = (FMT == MXQ_FMT_MXFP8) ? 8 : 2;
    constexpr uint32_t c_mant = (FMT == MXQ_FMT_MXFP8) ? 0x60u : 0x40u;  // .75 / .5 in 7 bits
    const uint32_t E = amax_bits >> 7;
    if (E == 0)
        return -127;
    int e = (int)E - 127 - k + ((amax_bits & 0x7Fu) > c_mant ? 1 : 0);
    return e < -127 ? -127 : (e > 127 ? 127 : e);
}

// The block's 16 words -> its codes (8 words of E4M3, or 4 of E2M1 pairs in o[0..3])
// and its scale byte (returned); `amax`: the largest magnitude's bf16 bits, 0x7F80 or
// above where a value is Inf or NaN.
template <int FMT>
__device__ __forceinline__ uint32_t mx_quantize_block(const uint32_t (&w)[16], uint32_t &amax, uint32_t (&o)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j)
        m = absmax_bf16x2(m, w[j]);
    amax = fold_halves(m);
    const int e = mx_exponent<FMT>(amax);
    const float sc = __uint_as_float((uint32_t)(127 - e) << 23);   // 2^-e, normal
    const float2 sc2 = make_float2(sc, sc);
    float2 y[16];
#pragma unroll
    for (int j = 0; j < 16; ++j)
        y[j] = __fmul2_rn(make_float2(bf16_lo(w[j]), bf16_hi(w[j])), sc2);
    if (FMT == MXQ_FMT_MXFP8) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            o[j] = e4m3x2(y[2 * j].x, y[2 * j].y) | (e4m3x2(y[2 * j + 1].x, y[2 * j + 1].y) << 16);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o[j] = e2m1x8(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
    }
    return (uint32_t)(e + 127);
}

// The same of an MXFP8 block that two neighbouring lanes hold, 8 words each, both of them
// together: each has its 16 codes, and both the scale byte and `amax`.
__device__ __forceinline__ uint32_t mx_quantize_half(uint4 v0, uint4 v1, uint32_t &amax, uint4 &o)
{
    const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        m = absmax_bf16x2(m, w[j]);
    m = fold_halves(m);
    amax = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    const int e = mx_exponent<MXQ_FMT_MXFP8>(amax);
    const float sc = __uint_as_float((uint32_t)(127 - e) << 23);   // 2^-e, normal
    const float2 sc2 = make_float2(sc, sc);
    uint32_t c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float2 y = __fmul2_rn(make_float2(bf16_lo(w[j]), bf16_hi(w[j])), sc2);
        c[j] = e4m3x2(y.x, y.y);
    }
    o = make_uint4(c[0] | (c[1] << 16), c[2] | (c[3] << 16), c[4] | (c[5] << 16), c[6] | (c[7] << 16));
    return (uint32_t)(e + 127);
}

} // namespace mxq
