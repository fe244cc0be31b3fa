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
// comes out.  A unit is 16 values of a token for the writer, 8 for the reader, whose
// neighbouring threads then write neighbouring 16 bytes.  A CTA has a run of tokens, and a
// thread the same unit of several of them (PER at a time, their loads together), so
// that what belongs to the unit (its head, its scale, its addresses) is worked out once.
// Where a token lies is a chain of four loads (its sequence, its length, its page): the
// threads look it up once for each of the CTA's tokens, and the writer has its first
// data on their way meanwhile.
//
// The reader moves bytes: 24 sequences of up to 8192 tokens, 4 heads of 128, 258 MB with
// MXFP8 in 48 us (82 % of a plain copy's rate; 59 with a look-up for each unit), 218 MB
// with NVFP4 in 42 us.  The writer of NVFP4 waits for itself: a thread has a block of 16
// and, with 4/6, two scales for it, and a quarter of the SM's warps are not enough to hide that
// chain (issue slots 53 % full).  17000 tokens of 8 heads take about 36 us (4/6), 25 (RTN);
// MXFP8 21 us.
#include "mx_block.cuh"
#include "mxq_cache.cuh"
#include "mxq_internal.h"
#include "nvfp4_block.cuh"

namespace mxq {

namespace {

constexpr uint32_t kWriteUnit = 16, kReadUnit = 8;
constexpr uint32_t kMostRows = 128;     // of a CTA

// How a CTA's threads divide its tokens.
struct Split {
    uint32_t T, rows;                   // rows (tokens): all; of a CTA
    uint32_t per;                       // units of a row, both tensors'
    uint32_t pass;                      // rows at a time
    FastDiv perdiv, headdiv;            // units of a row; units of a head
};

struct WriteArgs {
    CacheView c;
    const uint16_t *k, *v;
    int64_t k_stride, v_stride;         // values from one token to the next
    Split s;
};

struct ReadArgs {
    CacheView c;
    uint16_t *k, *v;
    Split s;
};

constexpr uint64_t kNowhere = ~0ull;

// Unit `in` of a row.
struct Unit {
    uint32_t head, at;                  // and its number in the head
    bool value;
};
__device__ __forceinline__ Unit unit_at(uint32_t in, const Split &s)
{
    Unit u;
    u.value = in >= s.per / 2u;
    in -= u.value ? s.per / 2u : 0u;
    u.head = fastdiv(in, s.headdiv);
    u.at = in - u.head * s.headdiv.d;
    return u;
}

// Places of the CTA's rows (kNowhere: none), by all threads.  The first CTA looks at every
// sequence's rows, for those that are none of the call's are no row's here.
__device__ __forceinline__ void find_places(const CacheView &c, uint32_t row0, uint32_t n, uint32_t T, uint64_t (&place)[kMostRows])
{
    if (blockIdx.x == 0)
        for (uint32_t b = threadIdx.x; b < c.seqs; b += blockDim.x) {
            uint32_t first;
            new_tokens(c, b, T, first);
        }
    for (uint32_t i0 = threadIdx.x & ~31u; i0 < n; i0 += blockDim.x) {
        const uint32_t i = i0 + (threadIdx.x & 31u);
        uint64_t at;
        const bool ok = find_place(c, row0 + min(i, n - 1u), T, at);
        if (i < n)
            place[i] = ok ? at : kNowhere;
    }
    __syncthreads();
}

} // namespace

template <int FMT, bool FOUR_SIX, int PER>
__global__ void __launch_bounds__(256, 3) cache_write_kernel(const WriteArgs a)
{
    constexpr bool fp4 = FMT == MXQ_FMT_NVFP4;
    __shared__ uint64_t place[kMostRows];
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();
    const uint32_t row0 = blockIdx.x * a.s.rows, rows = min(a.s.rows, a.s.T - row0);
    const uint32_t off = fastdiv(threadIdx.x, a.s.perdiv);
    bool looked = false;
    // Every lane takes every turn (lanes share a block's maximum): `live` has units left.
    for (uint32_t in0 = 0; in0 < a.s.per; in0 += blockDim.x) {
        const uint32_t in = in0 + threadIdx.x - off * a.s.per;
        const bool live = off < a.s.pass && in < a.s.per;
        const Unit u = unit_at(live ? in : 0u, a.s);
        const int64_t stride = u.value ? a.v_stride : a.k_stride;
        const uint16_t *src = (u.value ? a.v : a.k) + (int64_t)row0 * stride + (u.head * a.s.headdiv.d + u.at) * kWriteUnit;
        uint8_t *codes = u.value ? a.c.v_codes : a.c.k_codes, *scales = u.value ? a.c.v_scales : a.c.k_scales;
        const uint64_t before = ((uint64_t)u.head << a.c.page_log) * a.s.headdiv.d + u.at;
        GroupConst gc;
        bool good = true;
        if constexpr (fp4) {
            const float s2 = __ldg((u.value ? a.c.v_s2 : a.c.k_s2) + u.head);
            good = s2 >= 0.0f && s2 < INFINITY;
            gc = make_group_const_from_s2(s2);
        }
        for (uint32_t r0 = 0; r0 < rows; r0 += PER * a.s.pass) {
            uint4 v[PER][2];
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const uint32_t r = min(r0 + i * a.s.pass + off, rows - 1u);
                const uint4 *p = reinterpret_cast<const uint4 *>(src + r * stride);
                v[i][0] = __ldg(p);
                v[i][1] = __ldg(p + 1);
            }
            if (!looked)
                find_places(a.c, row0, rows, a.s.T, place);
            looked = true;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const uint32_t r = r0 + i * a.s.pass + off;
                const uint64_t at = live && r < rows ? place[r] : kNowhere;
                const uint64_t b = at * a.s.headdiv.d + before;     // number of the unit
                if constexpr (fp4) {
                    if (at == kNowhere)
                        continue;
                    if (!good) {
                        atomicOr(a.c.status, MXQ_DEV_INVALID_SCALE);
                        continue;
                    }
                    const BlockOut o = quantize_block<FOUR_SIX>(v[i][0], v[i][1], gc);
                    if (!(o.amax < INFINITY))
                        atomicOr(a.c.status, MXQ_DEV_NONFINITE_INPUT);
                    reinterpret_cast<uint2 *>(codes)[b] = o.codes;
                    scales[b] = (uint8_t)o.scale;
                } else {
                    uint32_t amax;
                    uint4 o;
                    const uint32_t e = mx_quantize_half(v[i][0], v[i][1], amax, o);
                    if (at == kNowhere)
                        continue;
                    if (amax >= 0x7F80u)
                        atomicOr(a.c.status, MXQ_DEV_NONFINITE_INPUT);
                    reinterpret_cast<uint4 *>(codes)[b] = o;
                    if ((u.at & 1u) == 0u)
                        scales[b >> 1] = (uint8_t)e;
                }
            }
        }
    }
}

// 8 codes -> 16 bytes of bf16.  MXFP8: q 2^e, exact unless it leaves bf16's normal
// numbers; NVFP4: RN_bf16(RN32((q D) s2)).
template <int FMT, int PER>
__global__ void __launch_bounds__(256) cache_read_kernel(const ReadArgs a)
{
    constexpr bool fp4 = FMT == MXQ_FMT_NVFP4;
    constexpr int block = fp4 ? 2 : 4;      // units of a block
    __shared__ uint64_t place[kMostRows];
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();
    const uint32_t row0 = blockIdx.x * a.s.rows, rows = min(a.s.rows, a.s.T - row0);
    const uint32_t off = fastdiv(threadIdx.x, a.s.perdiv);
    find_places(a.c, row0, rows, a.s.T, place);
    if (off >= a.s.pass)
        return;
    for (uint32_t in = threadIdx.x - off * a.s.per; in < a.s.per; in += blockDim.x) {
        const Unit u = unit_at(in, a.s);
        const uint8_t *codes = u.value ? a.c.v_codes : a.c.k_codes, *scales = u.value ? a.c.v_scales : a.c.k_scales;
        const uint64_t before = ((uint64_t)u.head << a.c.page_log) * a.s.headdiv.d + u.at;
        uint4 *dst = reinterpret_cast<uint4 *>(u.value ? a.v : a.k) + (uint64_t)row0 * (a.s.per / 2u) +
                     u.head * a.s.headdiv.d + u.at;
        const float s2 = fp4 ? __ldg((u.value ? a.c.v_s2 : a.c.k_s2) + u.head) : 1.0f;
        for (uint32_t r0 = off; r0 < rows; r0 += PER * a.s.pass) {
            uint2 w[PER];
            uint32_t sc[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const uint32_t r = r0 + i * a.s.pass;
                const uint64_t at = r < rows ? place[r] : kNowhere, b = at * a.s.headdiv.d + before;    // number of the unit
                sc[i] = 256u;           // no place
                if (at == kNowhere)
                    continue;
                if (fp4)
                    w[i] = make_uint2(__ldg(reinterpret_cast<const uint32_t *>(codes) + b), 0u);
                else
                    w[i] = __ldg(reinterpret_cast<const uint2 *>(codes) + b);
                sc[i] = __ldg(scales + b / block);
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (sc[i] > 255u)
                    continue;
                uint32_t h[4], o[4];
                float d;
                if constexpr (fp4) {
                    e2m1x8_to_f16x2(w[i].x, h);
                    d = f16x2_to_float2(e4m3x2_to_f16x2(sc[i])).x;
                } else {
                    h[0] = e4m3x2_to_f16x2(w[i].x);
                    h[1] = e4m3x2_to_f16x2(w[i].x >> 16);
                    h[2] = e4m3x2_to_f16x2(w[i].y);
                    h[3] = e4m3x2_to_f16x2(w[i].y >> 16);
                    d = sc[i] == 255u ? __uint_as_float(0x7FC00000u) : sc[i] ? __uint_as_float(sc[i] << 23) : 0x1p-127f;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float2 q = __fmul2_rn(f16x2_to_float2(h[j]), make_float2(d, d));
                    if (fp4)
                        q = __fmul2_rn(q, make_float2(s2, s2));
                    const __nv_bfloat162 r = __floats2bfloat162_rn(q.x, q.y);
                    o[j] = *reinterpret_cast<const uint32_t *>(&r);
                }
                dst[(uint64_t)(r0 + i * a.s.pass) * (a.s.per / 2u)] = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
    }
}

namespace {

// Threads for a row's units, 256 at most: some whole rows, or an even share of one.
uint32_t split(Split &s, const CacheView &c, int dim, uint32_t unit, uint32_t T)
{
    s.T = T;
    s.per = 2u * c.heads * ((uint32_t)dim / unit);
    s.pass = s.per <= 256u ? 256u / s.per : 1u;
    s.perdiv = make_fastdiv(s.per);
    s.headdiv = make_fastdiv((uint32_t)dim / unit);
    const uint32_t parts = (s.per + 255u) / 256u, threads = s.per <= 256u ? s.pass * s.per : (s.per + parts - 1u) / parts;
    return (threads + 31u) / 32u * 32u;
}

// One row a thread where that does not fill the card (2048 threads an SM): the shortest
// way through; `PER` where it does.
template <int PER, typename K1, typename KN, typename A>
cudaError_t go(K1 one, KN several, A &a, uint32_t threads, cudaStream_t s)
{
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return e;
    const bool few = (uint64_t)a.s.T * a.s.per <= (uint64_t)sms * 2048u;
    a.s.rows = a.s.pass * (few ? 1u : (uint32_t)PER);
    return launch_dependent(few ? one : several, dim3((a.s.T + a.s.rows - 1u) / a.s.rows), threads, 0, s, a);
}

} // namespace

cudaError_t launch_cache_write(const CacheView &c, int fmt, int dim, int four_six, const uint16_t *k, int64_t k_stride,
                               const uint16_t *v, int64_t v_stride, uint32_t T, cudaStream_t s)
{
    WriteArgs a;
    a.c = c;
    a.k = k;
    a.v = v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    const uint32_t threads = split(a.s, c, dim, kWriteUnit, T);
    if (fmt == MXQ_FMT_MXFP8)
        return go<4>(cache_write_kernel<MXQ_FMT_MXFP8, false, 1>, cache_write_kernel<MXQ_FMT_MXFP8, false, 4>, a, threads, s);
    if (four_six)
        return go<4>(cache_write_kernel<MXQ_FMT_NVFP4, true, 1>, cache_write_kernel<MXQ_FMT_NVFP4, true, 4>, a, threads, s);
    return go<4>(cache_write_kernel<MXQ_FMT_NVFP4, false, 1>, cache_write_kernel<MXQ_FMT_NVFP4, false, 4>, a, threads, s);
}

cudaError_t launch_cache_read(const CacheView &c, int fmt, int dim, uint32_t T, uint16_t *k, uint16_t *v,
                              cudaStream_t s)
{
    ReadArgs a;
    a.c = c;
    a.k = k;
    a.v = v;
    const uint32_t threads = split(a.s, c, dim, kReadUnit, T);
    if (fmt == MXQ_FMT_MXFP8)
        return go<8>(cache_read_kernel<MXQ_FMT_MXFP8, 1>, cache_read_kernel<MXQ_FMT_MXFP8, 8>, a, threads, s);
    return go<8>(cache_read_kernel<MXQ_FMT_NVFP4, 1>, cache_read_kernel<MXQ_FMT_NVFP4, 8>, a, threads, s);
}

} // namespace mxq
