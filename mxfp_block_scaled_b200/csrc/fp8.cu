// fp8.cu -- block-FP8 quantization: E4M3 values with one fp32 scale per
// 1 x 128 (token tiles) or 128 x 128 (weights) block (sm_100a).
//
// Method (the format mxq_requant_fp8_mx reads): scale = RN32(amax / 448),
// code = E4M3(RN32(x / scale)), round to nearest even, saturating; a block
// whose amax is 0 has scale 0 and codes 0.  amax of a non-zero bf16 block is
// at least 2^-133, so its scale is never rounded to 0.
//
// Both kernels read x once into registers, so HBM is the bound: 2 B in,
// 1 B out and a scale per block.  The quotient is a correctly rounded
// reciprocal of the scale and one FMA correction (div2_bf16) while the scale
// lies in [2^-60, 2^60]; there the quotient is the IEEE one, except where it
// is so small (below 2^-60) that its code is a signed 0 either way.  Outside
// that range the IEEE division is called.
#include "mxq_device.cuh"
#include "mxq_internal.h"
#include "mxq.h"

namespace mxq {

// Eight bf16 (four words) of a block with scale d and reciprocal r -> eight
// E4M3 codes.
__device__ __forceinline__ uint2 fp8_codes8(const uint4 &v, float d, float r, bool mid)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t h[4];
    if (mid) {
        const float2 dd = make_float2(d, d), nr = make_float2(-r, -r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 y = div2_bf16(make_float2(bf16_lo(w[i]), bf16_hi(w[i])), dd, nr);
            h[i] = e4m3x2(y.x, y.y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            h[i] = d > 0.0f ? e4m3x2(__fdiv_rn(bf16_lo(w[i]), d), __fdiv_rn(bf16_hi(w[i]), d)) : 0u;
    }
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

__device__ __forceinline__ uint32_t absmax8(const uint4 &v)
{
    uint32_t m = absmax_bf16x2(0u, v.x);
    m = absmax_bf16x2(m, v.y);
    m = absmax_bf16x2(m, v.z);
    return fold_halves(absmax_bf16x2(m, v.w));
}

// Scale of a block from the bits of its amax; r is its reciprocal where mid.
__device__ __forceinline__ float fp8_scale(uint32_t amax_bits, float &r, bool &mid)
{
    const float d = __fdiv_rn(__uint_as_float(amax_bits << 16), 448.0f);
    mid = d >= 0x1p-60f && d <= 0x1p60f;
    r = mid ? rcp_rn_mid(d) : 0.0f;
    return d;
}

// 1 x 128 blocks: 8 lanes hold one, 16 values each (two loads of 16 bytes, half
// a block apart), so that the scale's division and reciprocal are shared by
// 16 values (with 8 values a lane they took as long as the memory: 75.7 us for
// 65536 x 2048 values, 60.7 us so: 6.7 TB/s).  A thread takes kRowUnroll blocks.
template <int kRowUnroll>
__global__ void __launch_bounds__(256)
fp8_row_kernel(const uint16_t *__restrict__ x, uint32_t nblk, uint32_t cols, const FastDiv nbc,
               uint8_t *__restrict__ codes, float *__restrict__ scales, uint32_t *__restrict__ status)
{
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();
    const uint32_t l8 = (threadIdx.x & 7u) * 8u;
    // every lane of a warp runs the same steps (the reductions below name all
    // 32 lanes); blocks past the end hold zeros and are not stored
    const uint64_t b0 = (uint64_t)blockIdx.x * (32u * kRowUnroll) + (threadIdx.x >> 3);
    uint4 v[kRowUnroll][2];
    uint64_t at[kRowUnroll];
    bool in[kRowUnroll][2];
    uint32_t bad = 0;
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
        const uint32_t b = (uint32_t)(b0 + 32u * u), row = fastdiv(b, nbc), c = (b - row * nbc.d) * 128u + l8;
        at[u] = (uint64_t)row * cols + c;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            in[u][h] = b0 + 32u * u < nblk && c + 64u * h < cols;
            v[u][h] = in[u][h] ? __ldg(reinterpret_cast<const uint4 *>(x + at[u] + 64 * h)) : make_uint4(0u, 0u, 0u, 0u);
        }
    }
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
        uint32_t m = max(absmax8(v[u][0]), absmax8(v[u][1]));
#pragma unroll
        for (int o = 4; o > 0; o >>= 1)
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        bad |= m >= 0x7F80u;
        float r;
        bool mid;
        const float d = fp8_scale(m, r, mid);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (in[u][h])
                *reinterpret_cast<uint2 *>(codes + at[u] + 64 * h) = fp8_codes8(v[u][h], d, r, mid);
        if (in[u][0] && l8 == 0)
            scales[b0 + 32u * u] = d;
    }
    if (bad)
        atomicOr(status, MXQ_DEV_NONFINITE_INPUT);
}

// 128 x 128 blocks: one CTA of 256 threads holds one in registers (64 values
// a thread), so x is read once although the amax spans 128 rows.
__global__ void __launch_bounds__(256)
fp8_block_kernel(const uint16_t *__restrict__ x, uint32_t rows, uint32_t cols, uint32_t nbc,
                 uint8_t *__restrict__ codes, float *__restrict__ scales, uint32_t *__restrict__ status)
{
    __shared__ uint32_t part[8];
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();
    const uint32_t br = blockIdx.x / nbc, bc = blockIdx.x - br * nbc;
    const uint32_t c = bc * 128u + (threadIdx.x & 15u) * 8u, r0 = br * 128u + (threadIdx.x >> 4);
    uint4 v[8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = r0 + 16u * i < rows && c < cols
                   ? __ldg(reinterpret_cast<const uint4 *>(x + (uint64_t)(r0 + 16u * i) * cols + c))
                   : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = max(m, absmax8(v[i]));
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((threadIdx.x & 31u) == 0)
        part[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = max(m, part[i]);
    float r;
    bool mid;
    const float d = fp8_scale(m, r, mid);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (r0 + 16u * i < rows && c < cols)
            *reinterpret_cast<uint2 *>(codes + (uint64_t)(r0 + 16u * i) * cols + c) = fp8_codes8(v[i], d, r, mid);
    if (threadIdx.x == 0) {
        scales[blockIdx.x] = d;
        if (m >= 0x7F80u)
            atomicOr(status, MXQ_DEV_NONFINITE_INPUT);
    }
}

cudaError_t launch_quantize_fp8(const uint16_t *x, int64_t rows, int64_t cols, int64_t brows, uint8_t *codes,
                                float *scales, uint32_t *status, cudaStream_t s)
{
    const uint32_t nbc = (uint32_t)((cols + 127) / 128);
    if (brows == 1) {
        const uint64_t nblk = (uint64_t)rows * nbc;
        // Two blocks a thread where every SM is full several times over (60.7
        // against 62.2 us above), one below (a token of 2048: 1.4 against 1.7 us).
        if (nblk > 1u << 16)
            return launch_dependent(fp8_row_kernel<2>, dim3((unsigned)((nblk + 63) / 64)), 256, 0, s, x, (uint32_t)nblk,
                                    (uint32_t)cols, make_fastdiv(nbc), codes, scales, status);
        return launch_dependent(fp8_row_kernel<1>, dim3((unsigned)((nblk + 31) / 32)), 256, 0, s, x, (uint32_t)nblk,
                                (uint32_t)cols, make_fastdiv(nbc), codes, scales, status);
    }
    const uint64_t grid = (uint64_t)((rows + 127) / 128) * nbc;
    return launch_dependent(fp8_block_kernel, dim3((unsigned)grid), 256, 0, s, x, (uint32_t)rows, (uint32_t)cols, nbc,
                            codes, scales, status);
}

} // namespace mxq
