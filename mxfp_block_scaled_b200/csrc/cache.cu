// cache.cu -- a key/value cache that is quantized as it is written and read
// back (sm_100a).
//
// The cache holds its tokens in pages: codes [pages, kv_heads, page_tokens,
// head_dim] of keys and of values, and a scale for each 32 (MXFP8) or 16
// (NVFP4) values of a head's row, [pages, kv_heads, page_tokens, head_dim /
// block].  A block is quantized exactly as the tensor quantizers do it
// (mx_block.cuh, nvfp4_block.cuh; NVFP4 with a given global scale for each head),
// so what is held does not depend on which of them wrote it.
//
// Both kernels are elementwise: one read of what is there, one write of what
// comes out.  A thread of the writer takes a block, a thread of the reader 16
// codes; neighbouring threads take neighbouring parts of a token's heads.
#include "mx_block.cuh"
#include "mxq_cache.cuh"
#include "mxq_internal.h"
#include "nvfp4_block.cuh"

namespace mxq {

namespace {

struct WriteArgs {
    CacheView c;
    const uint16_t *k, *v;
    int64_t k_stride, v_stride;         // values from one token to the next
    uint32_t T;
    uint64_t units;                     // threads that have a block
    FastDiv perdiv, blkdiv;             // blocks of a token (both tensors); blocks of a head
};

struct ReadArgs {
    CacheView c;
    uint16_t *k, *v;
    uint32_t T;
    uint64_t units;
    FastDiv perdiv, blkdiv;
};

// Thread `u` -> its token's row, tensor, head and block of the head.
struct Unit {
    uint32_t row, head, blk;
    bool value;
};
__device__ __forceinline__ Unit unit_at(uint64_t u, const FastDiv &perdiv, const FastDiv &blkdiv)
{
    Unit r;
    r.row = u >> 32 ? (uint32_t)(u / perdiv.d) : fastdiv((uint32_t)u, perdiv);
    uint32_t in = (uint32_t)(u - (uint64_t)r.row * perdiv.d);
    r.value = in >= perdiv.d / 2u;
    in -= r.value ? perdiv.d / 2u : 0u;
    r.head = fastdiv(in, blkdiv);
    r.blk = in - r.head * blkdiv.d;
    return r;
}

} // namespace

template <int FMT, bool FOUR_SIX>
__global__ void __launch_bounds__(256) cache_write_kernel(const WriteArgs a)
{
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();
    const uint64_t u = (uint64_t)blockIdx.x * 256u + threadIdx.x;
    if (u >= a.units)
        return;
    const Unit n = unit_at(u, a.perdiv, a.blkdiv);
    uint64_t at;
    if (!find_place(a.c, n.row, at))
        return;
    at += (uint64_t)n.head << a.c.page_log;
    constexpr uint32_t block = FMT == MXQ_FMT_NVFP4 ? 16u : 32u;
    const uint16_t *src = (n.value ? a.v + (int64_t)n.row * a.v_stride : a.k + (int64_t)n.row * a.k_stride) +
                          (n.head * a.blkdiv.d + n.blk) * block;
    uint8_t *codes = n.value ? a.c.v_codes : a.c.k_codes, *scales = n.value ? a.c.v_scales : a.c.k_scales;
    const uint64_t b = at * a.blkdiv.d + n.blk;         // number of the block
    uint4 v[block / 8];
#pragma unroll
    for (uint32_t i = 0; i < block / 8; ++i)
        v[i] = __ldg(reinterpret_cast<const uint4 *>(src) + i);
    if constexpr (FMT == MXQ_FMT_NVFP4) {
        const float s2 = __ldg((n.value ? a.c.v_s2 : a.c.k_s2) + n.head);
        if (!(s2 >= 0.0f && s2 < INFINITY)) {
            atomicOr(a.c.status, MXQ_DEV_INVALID_SCALE);
            return;
        }
        const BlockOut o = quantize_block<FOUR_SIX>(v[0], v[1], make_group_const_from_s2(s2));
        if (!(o.amax < INFINITY))
            atomicOr(a.c.status, MXQ_DEV_NONFINITE_INPUT);
        reinterpret_cast<uint2 *>(codes)[b] = o.codes;
        scales[b] = (uint8_t)o.scale;
    } else {
        const uint32_t w[16] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w,
                                v[2].x, v[2].y, v[2].z, v[2].w, v[3].x, v[3].y, v[3].z, v[3].w};
        uint32_t o[8], amax;
        scales[b] = (uint8_t)mx_quantize_block<FMT>(w, amax, o);
        if (amax >= 0x7F80u)
            atomicOr(a.c.status, MXQ_DEV_NONFINITE_INPUT);
        uint4 *dst = reinterpret_cast<uint4 *>(codes) + b * 2;
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

// 16 codes -> 32 bytes of bf16.  MXFP8: q 2^e, exact unless it leaves bf16's normal
// numbers; NVFP4: RN_bf16(RN32((q D) s2)).
template <int FMT>
__global__ void __launch_bounds__(256) cache_read_kernel(const ReadArgs a)
{
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();
    const uint64_t u = (uint64_t)blockIdx.x * 256u + threadIdx.x;
    if (u >= a.units)
        return;
    const Unit n = unit_at(u, a.perdiv, a.blkdiv);
    uint64_t at;
    if (!find_place(a.c, n.row, at))
        return;
    at += (uint64_t)n.head << a.c.page_log;
    const uint64_t b = at * a.blkdiv.d + n.blk;         // number of the 16 codes
    const uint8_t *codes = n.value ? a.c.v_codes : a.c.k_codes, *scales = n.value ? a.c.v_scales : a.c.k_scales;
    uint32_t h[8];
    float d, s2 = 1.0f;
    if constexpr (FMT == MXQ_FMT_NVFP4) {
        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(codes) + b);
        const uint32_t s = scales[b];
        e2m1x8_to_f16x2(w.x, *reinterpret_cast<uint32_t(*)[4]>(&h[0]));
        e2m1x8_to_f16x2(w.y, *reinterpret_cast<uint32_t(*)[4]>(&h[4]));
        d = f16x2_to_float2(e4m3x2_to_f16x2(s)).x;
        s2 = __ldg((n.value ? a.c.v_s2 : a.c.k_s2) + n.head);
    } else {
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(codes) + b);
        const uint32_t s = scales[b >> 1], q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[2 * i] = e4m3x2_to_f16x2(q[i]);
            h[2 * i + 1] = e4m3x2_to_f16x2(q[i] >> 16);
        }
        d = s == 255u ? __uint_as_float(0x7FC00000u) : s ? __uint_as_float(s << 23) : 0x1p-127f;
    }
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 q = f16x2_to_float2(h[i]);
        const __nv_bfloat162 r = __floats2bfloat162_rn(__fmul_rn(__fmul_rn(q.x, d), s2), __fmul_rn(__fmul_rn(q.y, d), s2));
        o[i] = *reinterpret_cast<const uint32_t *>(&r);
    }
    uint4 *dst = reinterpret_cast<uint4 *>(n.value ? a.v : a.k) +
                 ((uint64_t)n.row * a.c.heads + n.head) * (a.blkdiv.d * 2u) + n.blk * 2u;
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

cudaError_t launch_cache_write(const CacheView &c, int fmt, int dim, int four_six, const uint16_t *k, int64_t k_stride,
                               const uint16_t *v, int64_t v_stride, uint32_t T, cudaStream_t s)
{
    WriteArgs a;
    a.c = c;
    a.k = k;
    a.v = v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.T = T;
    const uint32_t blocks = (uint32_t)dim / (fmt == MXQ_FMT_NVFP4 ? 16u : 32u), per = 2u * c.heads * blocks;
    a.units = (uint64_t)T * per;
    a.perdiv = make_fastdiv(per);
    a.blkdiv = make_fastdiv(blocks);
    const dim3 grid((unsigned)((a.units + 255) / 256));
    if (fmt == MXQ_FMT_MXFP8)
        return launch_dependent(cache_write_kernel<MXQ_FMT_MXFP8, false>, grid, 256, 0, s, a);
    if (four_six)
        return launch_dependent(cache_write_kernel<MXQ_FMT_NVFP4, true>, grid, 256, 0, s, a);
    return launch_dependent(cache_write_kernel<MXQ_FMT_NVFP4, false>, grid, 256, 0, s, a);
}

cudaError_t launch_cache_read(const CacheView &c, int fmt, int dim, uint32_t T, uint16_t *k, uint16_t *v,
                              cudaStream_t s)
{
    ReadArgs a;
    a.c = c;
    a.k = k;
    a.v = v;
    a.T = T;
    const uint32_t parts = (uint32_t)dim / 16u, per = 2u * c.heads * parts;
    a.units = (uint64_t)T * per;
    a.perdiv = make_fastdiv(per);
    a.blkdiv = make_fastdiv(parts);
    const dim3 grid((unsigned)((a.units + 255) / 256));
    if (fmt == MXQ_FMT_MXFP8)
        return launch_dependent(cache_read_kernel<MXQ_FMT_MXFP8>, grid, 256, 0, s, a);
    return launch_dependent(cache_read_kernel<MXQ_FMT_NVFP4>, grid, 256, 0, s, a);
}

} // namespace mxq
