// linear.cu -- product of a few tokens with a block-scaled weight matrix
// (sm_100a):
//
//   y[t, n] = sum over blocks b of s[n, b] sum_{k in b} q[n, k] x[t, k]   (NVFP4: times s2)
//
// with codes q and scales s as the quantizers write them.  Few tokens share the
// read of the weights, which is the work: HBM is the bound and the arithmetic only
// has to keep out of its way.
//
// linear_rows_kernel brings the tokens into f16 rows times a power of two of the
// row (as the layer's, moe.cu: exact above 2^-31 of the row's largest element).
// linear_kernel: a task is 16 rows of w over the whole length K; a CTA of 8 warps
// takes a contiguous run of tasks, its warps one after the other, with up to 32
// token rows in shared memory.  A warp streams its tasks' codes and scales through
// its own ring of two chunks (16 rows of 256 bytes) with cp.async; with few tasks
// 2, 4 or 8 warps split K and add their sums in a fixed order.  mma.sync
// m16n8k16, f16 operands, fp32 sums: 16 weight rows by 8 tokens.  E2M1 and E4M3
// values, and E2M1 times an E4M3 scale, are exact in f16; UE8M0 scales multiply
// the fp32 sum of their 32 values.
#include "mxq_device.cuh"
#include "mxq_layer.h"
#include "mxq_mma.cuh"
#include "mxq.h"
#include <algorithm>

namespace mxq {

namespace {

constexpr int kWarps = 8;
constexpr uint32_t kThreads = 32 * kWarps;
// One chunk in shared memory: 16 rows of 256 bytes of codes, 272 apart, and the
// rows' scales, 48 apart: the fragment loads touch every bank once.
constexpr uint32_t kChunk = 256, kPitch = kChunk + 16, kScaleAt = 16 * kPitch, kScalePitch = 48;
constexpr uint32_t kSlot = kScaleAt + 16 * kScalePitch, kRing = 2 * kSlot;
constexpr uint32_t kPart = 16 * 32 * 4;        // a warp's sums: 16 rows by up to 32 tokens

struct Args {
    const uint32_t *xh;         // f16 rows [T, K], in the order of the fragments
    const float *xf;            // inverse factor of each
    const uint8_t *codes, *scales;
    const float *s2;
    void *y;
    uint32_t T, N, K;
    uint32_t row_bytes, row_scales;     // of a row of w
    uint32_t tiles, chunks, kslog;
    uint32_t cap;               // tokens of a CTA
    uint32_t xstride;           // bytes of a staged row
    uint32_t direct;            // scales are read where they lie (rows of them are not 4- or 8-byte aligned)
    FastDiv griddiv;
};

template <int FMT>
struct Fmt {
    static constexpr bool fp4 = FMT != MXQ_FMT_MXFP8;
    static constexpr uint32_t group_bytes = fp4 ? 64 : 128;             // of 128 codes
    static constexpr uint32_t chunk_k = 128 * kChunk / group_bytes;     // values of a row in a chunk
    static constexpr uint32_t block = FMT == MXQ_FMT_NVFP4 ? 16 : 32;
    static constexpr uint32_t sbytes = 128 / block;                     // scale bytes of 128 values
};

// Where four values lie in a staged row: 4-bit formats in order, a lane's word holds
// 8 codes; 8-bit formats: a lane has one word (4 codes) of two neighbouring
// pieces, so of every 32 values the quads 0, 4, 1, 5, ... follow one another.
template <bool FP4>
__device__ __forceinline__ uint32_t staged(uint32_t k)
{
    const uint32_t q = (k >> 2) & 7u;
    return FP4 ? k : (k & ~31u) + ((q & 3u) * 2u + (q >> 2)) * 4u;
}

} // namespace

// A CTA brings one token into f16: its largest magnitude, then its values.
template <bool FP4>
__global__ void __launch_bounds__(256)
linear_rows_kernel(const uint16_t *__restrict__ x, uint32_t K, uint32_t *__restrict__ xh, float *__restrict__ xf,
                   uint32_t *__restrict__ status)
{
    __shared__ uint32_t part[8];
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();
    const uint16_t *src = x + (uint64_t)blockIdx.x * K;
    char *dst = reinterpret_cast<char *>(xh) + (uint64_t)blockIdx.x * K * 2u;
    uint32_t m = 0;
    for (uint32_t k = threadIdx.x * 8u; k < K; k += 2048u) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src + k));
        m = max(m, fold_halves(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(0u, v.x), v.y), v.z), v.w)));
    }
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((threadIdx.x & 31u) == 0)
        part[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = max(m, part[i]);
    m <<= 16;
    const float f = row_factor(m);
    if (threadIdx.x == 0) {
        xf[blockIdx.x] = 1.0f / f;
        if (m >= 0x7F800000u)
            atomicOr(status, MXQ_DEV_NONFINITE_INPUT);
    }
    for (uint32_t k = threadIdx.x * 8u; k < K; k += 2048u) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src + k));
        *reinterpret_cast<uint2 *>(dst + staged<FP4>(k) * 2u) =
            make_uint2(half2_bits(bf16_lo(v.x) * f, bf16_hi(v.x) * f), half2_bits(bf16_lo(v.y) * f, bf16_hi(v.y) * f));
        *reinterpret_cast<uint2 *>(dst + staged<FP4>(k + 4u) * 2u) =
            make_uint2(half2_bits(bf16_lo(v.z) * f, bf16_hi(v.z) * f), half2_bits(bf16_lo(v.w) * f, bf16_hi(v.w) * f));
    }
}

template <int FMT, int NT, typename Out>
__global__ void __launch_bounds__(kThreads, 2)
linear_kernel(const Args a)
{
    using F = Fmt<FMT>;
    extern __shared__ __align__(128) char smem[];
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5, g8 = lane >> 2, t4 = lane & 3u;
    char *ring = smem + warp * kRing;
    float *part = reinterpret_cast<float *>(smem + kWarps * kRing);
    char *xs = smem + kWarps * (kRing + kPart);
    const uint32_t ring_s = smem_addr(ring);
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();

    const uint32_t tok0 = blockIdx.y * a.cap, ntok = min(a.cap, a.T - tok0);
    const uint32_t t0 = fastdiv(a.tiles * blockIdx.x, a.griddiv), t1 = fastdiv(a.tiles * (blockIdx.x + 1u), a.griddiv);
    const uint32_t lg = a.kslog, ks = 1u << lg, teams = kWarps >> lg, team = warp >> lg, q = warp & (ks - 1u);
    const uint32_t c0 = (a.chunks * q) >> lg, c1 = (a.chunks * (q + 1u)) >> lg;

    // Token rows.
    for (uint32_t i = tid; i < ntok * (a.K / 8u); i += kThreads) {
        const uint32_t r = i / (a.K / 8u), p = i - r * (a.K / 8u);
        cp16(smem_addr(xs) + r * a.xstride + p * 16u, reinterpret_cast<const char *>(a.xh) + ((uint64_t)(tok0 + r) * a.K + p * 8u) * 2u);
    }
    cp_commit();

    const uint32_t piece = lane & 7u;
    constexpr uint32_t spieces = F::fp4 ? 4 : 2;            // scale pieces of a row of a chunk
    const uint32_t srow = lane / spieces, spiece = lane % spieces;
    uint32_t ptask = t0 + team, pch = c0;
    const uint8_t *pcode[4], *pscale[2];
    auto locate = [&]() {       // rows past the last are read as the last: their sums are not stored
        const uint32_t r0 = ptask * 16u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            pcode[i] = a.codes + (uint64_t)min(r0 + (lane >> 3) + 4u * i, a.N - 1u) * a.row_bytes + piece * 16u;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            pscale[i] = a.scales + (uint64_t)min(r0 + srow + 8u * i, a.N - 1u) * a.row_scales + spiece * F::sbytes;
    };
    auto issue = [&](uint32_t slot) {
        if (ptask < t1) {
            const uint32_t dst = ring_s + slot * kSlot + (lane >> 3) * kPitch + piece * 16u;
            const uint32_t left = a.row_bytes - pch * kChunk;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (piece * 16u + 128u * h < left)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        cp16(dst + 4 * i * kPitch + 128u * h, pcode[i] + (uint64_t)pch * kChunk + 128u * h);
            if (!a.direct && spiece * F::group_bytes < left) {
                const uint32_t sd = ring_s + slot * kSlot + kScaleAt + srow * kScalePitch + spiece * F::sbytes;
                const uint32_t at = pch * (kChunk / F::group_bytes) * F::sbytes;
                cp_small<F::sbytes>(sd, pscale[0] + at);
                if (F::fp4)             // 4 pieces a row: the lanes cover 8 rows
                    cp_small<F::sbytes>(sd + 8 * kScalePitch, pscale[1] + at);
            }
            if (++pch == c1) {
                pch = c0;
                ptask += teams;
                if (ptask < t1)
                    locate();
            }
        }
        cp_commit();
    };
    if (ptask < t1)
        locate();
    issue(0);
    cp_wait<1>();
    __syncthreads();

    uint32_t slot = 0;
    const char *xrow[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i)        // columns without a token read the first one's row; their sums are not stored
        xrow[i] = xs + (i * 8u + g8 < ntok ? i * 8u + g8 : 0u) * a.xstride + t4 * 16u;
    for (uint32_t task0 = t0; task0 < t1; task0 += teams) {
        const uint32_t task = task0 + team;
        float acc[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
            acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
        for (uint32_t ch = task < t1 ? c0 : c1; ch < c1; ++ch) {
            cp_wait<0>();
            __syncwarp();
            issue(slot ^ 1u);
            const char *cw = ring + slot * kSlot + g8 * kPitch + t4 * 4u;
            const char *sb = ring + slot * kSlot + kScaleAt + g8 * kScalePitch;
            slot ^= 1u;
            uint32_t k = ch * F::chunk_k;
            const uint32_t end = min(a.K, k + F::chunk_k);
            const uint8_t *ds0 = a.scales + (uint64_t)min(task * 16u + g8, a.N - 1u) * a.row_scales;
            const uint8_t *ds1 = a.scales + (uint64_t)min(task * 16u + g8 + 8u, a.N - 1u) * a.row_scales;
            for (; k < end; k += 128u, cw += F::group_bytes, sb += F::sbytes) {
                uint32_t w0[2], w1[2];          // the scales of 128 values of both rows
                if (!a.direct) {
                    if (F::sbytes == 8) {
                        const uint2 u = lds64(sb), v = lds64(sb + 8 * kScalePitch);
                        w0[0] = u.x, w0[1] = u.y, w1[0] = v.x, w1[1] = v.y;
                    } else {
                        w0[0] = lds32(sb);
                        w1[0] = lds32(sb + 8 * kScalePitch);
                    }
                } else {
                    w0[0] = w0[1] = w1[0] = w1[1] = 0u;
                    const uint32_t n = min(end - k, 128u) / F::block;
                    for (uint32_t i = 0; i < n; ++i) {
                        w0[i >> 2] |= (uint32_t)__ldg(ds0 + k / F::block + i) << (8u * (i & 3u));
                        w1[i >> 2] |= (uint32_t)__ldg(ds1 + k / F::block + i) << (8u * (i & 3u));
                    }
                }
                float d0[4], d1[4];
                uint32_t s0[4], s1[4];
                if (FMT == MXQ_FMT_NVFP4) {     // pairs of scales of 32 values, the one of this lane's 16 first
                    const uint32_t half8 = (t4 >> 1) * 8u;
                    e4m3x4_unpack(w0[0] >> half8, s0[0], s0[1]);
                    e4m3x4_unpack(w0[1] >> half8, s0[2], s0[3]);
                    e4m3x4_unpack(w1[0] >> half8, s1[0], s1[1]);
                    e4m3x4_unpack(w1[1] >> half8, s1[2], s1[3]);
                } else {
                    ue8m0x4(w0[0], d0);
                    ue8m0x4(w1[0], d1);
                }
#pragma unroll
                for (uint32_t u = 0; u < 4; ++u) {           // 32 values of a row
                    if (k + u * 32u >= end)
                        break;
                    uint32_t p0[4], p1[4];
                    if (F::fp4) {
                        e2m1x8_unpack(lds32(cw + u * 16u), p0);
                        e2m1x8_unpack(lds32(cw + u * 16u + 8 * kPitch), p1);
                    } else {
                        e4m3x4_unpack(lds32(cw + u * 32u), p0[0], p0[1]);
                        e4m3x4_unpack(lds32(cw + u * 32u + 16), p0[2], p0[3]);
                        e4m3x4_unpack(lds32(cw + u * 32u + 8 * kPitch), p1[0], p1[1]);
                        e4m3x4_unpack(lds32(cw + u * 32u + 8 * kPitch + 16), p1[2], p1[3]);
                    }
                    if (FMT == MXQ_FMT_NVFP4) {
                        const uint32_t e0 = low2(s0[u]), e1 = low2(s1[u]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            p0[i] = hmul2_bits(p0[i], e0);
                            p1[i] = hmul2_bits(p1[i], e1);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const uint4 b = lds128(xrow[i] + (k + u * 32u) * 2u);
                        if (FMT == MXQ_FMT_NVFP4) {
                            mma16816(acc[i], p0[0], p1[0], p0[1], p1[1], b.x, b.y);
                            mma16816(acc[i], p0[2], p1[2], p0[3], p1[3], b.z, b.w);
                        } else {
                            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                            mma16816(c, p0[0], p1[0], p0[1], p1[1], b.x, b.y);
                            mma16816(c, p0[2], p1[2], p0[3], p1[3], b.z, b.w);
                            acc[i][0] = fmaf(c[0], d0[u], acc[i][0]);
                            acc[i][1] = fmaf(c[1], d0[u], acc[i][1]);
                            acc[i][2] = fmaf(c[2], d1[u], acc[i][2]);
                            acc[i][3] = fmaf(c[3], d1[u], acc[i][3]);
                        }
                    }
                }
            }
        }
        if (ks > 1u) {          // the team's sums, in warp order
            float *mine = part + warp * (kPart / 4);
#pragma unroll
            for (int i = 0; i < NT; ++i)
                *reinterpret_cast<float4 *>(mine + (i * 32u + lane) * 4u) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
            named_barrier_sync(1 + (int)team, (int)(ks * 32u));
            if (q == 0)
                for (uint32_t w = 1; w < ks; ++w)
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const float4 v = *reinterpret_cast<const float4 *>(mine + w * (kPart / 4) + (i * 32u + lane) * 4u);
                        acc[i][0] += v.x;
                        acc[i][1] += v.y;
                        acc[i][2] += v.z;
                        acc[i][3] += v.w;
                    }
            named_barrier_sync(1 + (int)team, (int)(ks * 32u));
        }
        if (q == 0 && task < t1) {
            const float s2 = FMT == MXQ_FMT_NVFP4 ? __ldg(a.s2) : 1.0f;
            Out *y = static_cast<Out *>(a.y);
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j) {
                    const uint32_t t = i * 8u + t4 * 2u + (j & 1u), n = task * 16u + g8 + (j >> 1) * 8u;
                    if (t < ntok && n < a.N) {
                        const float v = acc[i][j] * s2 * __ldg(a.xf + tok0 + t);
                        if constexpr (sizeof(Out) == 2)
                            y[(uint64_t)(tok0 + t) * a.N + n] = __float2bfloat16_rn(v);
                        else
                            y[(uint64_t)(tok0 + t) * a.N + n] = v;
                    }
                }
        }
    }
    cp_wait<0>();
}

namespace {

constexpr size_t kSmemHalf = 113 * 1024, kSmemMax = 227 * 1024;

template <int FMT, int NT, typename Out>
cudaError_t go(const Args &a, dim3 grid, size_t smem, cudaStream_t s)
{
    const auto k = linear_kernel<FMT, NT, Out>;
    // always the largest, so that calls of other sizes from other threads set the same
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax);
    return e != cudaSuccess ? e : launch_dependent(k, grid, kThreads, smem, s, a);
}

template <int FMT>
cudaError_t plan(const LinearArgs &l, int out_f32, int sms, cudaStream_t s)
{
    using F = Fmt<FMT>;
    Args a;
    a.xh = l.xh;
    a.xf = l.xf;
    a.codes = l.codes;
    a.scales = l.scales;
    a.s2 = l.s2;
    a.y = l.y;
    a.T = (uint32_t)l.T;
    a.N = (uint32_t)l.N;
    a.K = (uint32_t)l.K;
    a.row_bytes = F::fp4 ? a.K / 2 : a.K;
    a.row_scales = a.K / F::block;
    a.tiles = (a.N + 15) / 16;
    a.chunks = (a.row_bytes + kChunk - 1) / kChunk;
    a.xstride = a.K * 2 + 64;           // 64 mod 128: rows of a fragment load fall on different banks
    a.direct = a.K % 128 != 0 || (reinterpret_cast<uintptr_t>(l.scales) % F::sbytes) != 0;
    const size_t fixed = (size_t)kWarps * (kRing + kPart);
    // As many tokens as fit, 32 at most, in groups of about the same size.
    const uint32_t most = (uint32_t)std::min<size_t>((kSmemMax - fixed) / a.xstride, 32);
    const uint32_t groups = (a.T + most - 1) / most;
    a.cap = (a.T + groups - 1) / groups;
    const size_t smem = fixed + (size_t)a.cap * a.xstride;
    const uint32_t ctas = (uint32_t)std::min<uint64_t>((uint64_t)sms * (smem <= kSmemHalf ? 2 : 1), a.tiles);
    a.griddiv = make_fastdiv(ctas);
    a.kslog = 0;
    while (a.kslog < 3 && (2u << a.kslog) <= a.chunks && ((uint64_t)a.tiles * 2 << a.kslog) <= (uint64_t)ctas * kWarps)
        ++a.kslog;
    cudaError_t e = launch_dependent(linear_rows_kernel<F::fp4>, dim3(a.T), 256, 0, s, l.x, a.K, l.xh, l.xf, l.status);
    if (e != cudaSuccess)
        return e;
    const dim3 grid(ctas, groups);
    const uint32_t nt = (a.cap + 7) / 8;
    if (out_f32)
        return nt == 1   ? go<FMT, 1, float>(a, grid, smem, s)
               : nt == 2 ? go<FMT, 2, float>(a, grid, smem, s)
                         : go<FMT, 4, float>(a, grid, smem, s);
    return nt == 1   ? go<FMT, 1, __nv_bfloat16>(a, grid, smem, s)
           : nt == 2 ? go<FMT, 2, __nv_bfloat16>(a, grid, smem, s)
                     : go<FMT, 4, __nv_bfloat16>(a, grid, smem, s);
}

} // namespace

size_t linear_rows_bytes(int64_t T, int64_t K) { return ((size_t)(T * K) * 2 + 255) / 256 * 256; }
size_t linear_workspace_bytes(int64_t T, int64_t K)
{
    return linear_rows_bytes(T, K) + ((size_t)T * 4 + 255) / 256 * 256;
}

cudaError_t launch_linear(const LinearArgs &l, int fmt, int out_f32, cudaStream_t s)
{
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return e;
    switch (fmt) {
    case MXQ_FMT_NVFP4: return plan<MXQ_FMT_NVFP4>(l, out_f32, sms, s);
    case MXQ_FMT_MXFP4: return plan<MXQ_FMT_MXFP4>(l, out_f32, sms, s);
    default: return plan<MXQ_FMT_MXFP8>(l, out_f32, sms, s);
    }
}

} // namespace mxq
