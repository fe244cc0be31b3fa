// linear.cu -- product of a few tokens with a block-scaled weight matrix
// (sm_100a):
//
//   y[t, n] = sum over blocks b of s[n, b] sum_{k in b} q[n, k] x[t, k]   (NVFP4: times s2)
//
// with codes q and scales s as the quantizers write them.  Few tokens share the
// read of the weights, which is the work: HBM is the bound and the arithmetic only
// has to keep out of its way.
//
// Tokens are brought into f16 rows times a power of two of the row (as the layer's,
// moe.cu: exact above 2^-31 of the row's largest element), by each CTA for itself where
// they are few, otherwise by linear_rows_kernel once for all.
// linear_kernel: a task is 16 rows of w over the whole length K; a CTA of 8 to 16 warps
// takes a contiguous run of tasks, its warps one after the other, with up to 32 token rows
// in shared memory.  A warp streams its tasks' codes and scales through its own ring of two
// or three chunks (16 rows of 128 bytes) with cp.async; with few tasks
// 2, 4 or 8 warps split K and add their sums in a fixed order.  mma.sync
// m16n8k16, f16 operands, fp32 sums: 16 weight rows by 8 tokens.  E2M1 and E4M3
// values, and E2M1 times an E4M3 scale, are exact in f16; UE8M0 scales multiply
// the fp32 sum of their 32 values.  The tensor core's own sums are cut to fp32 rather
// than rounded, so they run over 128 values at most (NVFP4) before an fp32 addition.
#include "mxq_device.cuh"
#include "mxq_layer.h"
#include "mxq_mma.cuh"
#include "mxq.h"
#include <algorithm>

namespace mxq {

namespace {

constexpr uint32_t kOwnTurns = 6;       // pieces of 8 values of a thread, of tokens that every CTA brings into f16 itself
constexpr uint32_t kMostWarps = 16, kMostSlots = 3, kMostCap = 32;
// One chunk in shared memory: 16 rows of 128 bytes of codes, and the rows' scales, 16 apart.
// The fragment loads touch every bank once: of 4 bytes (MX) with rows 144 apart, of 16
// (NVFP4) with the halves of every other row swapped.
constexpr uint32_t kChunk = 128, kScaleAt = 16 * (kChunk + 16), kScalePitch = 16;
constexpr uint32_t kSlot = kScaleAt + 16 * kScalePitch;

struct Args {
    const uint16_t *x;          // tokens, or null where linear_rows_kernel has them ready:
    const uint32_t *xh;         // f16 rows [T, width], in the order of the fragments
    const float *xf;            // inverse factor of each
    uint32_t *status;
    const uint8_t *codes, *scales;
    const float *s2;
    void *y;
    uint32_t T, N, K;
    uint32_t width;             // K rounded up to 128: a staged row ends with zeros
    uint32_t row_bytes, row_scales;     // of a row of w
    uint32_t tiles, chunks, kslog;
    uint32_t cap;               // tokens of a CTA
    uint32_t slots;             // of a warp's ring
    uint32_t xstride;           // bytes of a staged row
    uint32_t direct;            // scales are read where they lie (rows of them are not 4- or 8-byte aligned)
    uint32_t per, rest;         // tasks of a CTA, one more of the first `rest`
    FastDiv rowdiv;             // 16-byte pieces of a token
};

template <int FMT>
struct Fmt {
    static constexpr bool fp4 = FMT != MXQ_FMT_MXFP8, swap = FMT == MXQ_FMT_NVFP4;
    static constexpr uint32_t pitch = swap ? kChunk : kChunk + 16;
    static constexpr uint32_t group_bytes = fp4 ? 64 : 128;             // of 128 codes
    static constexpr uint32_t groups = kChunk / group_bytes;            // of a row in a chunk
    static constexpr uint32_t chunk_k = 128 * groups;                   // values
    static constexpr uint32_t block = FMT == MXQ_FMT_NVFP4 ? 16 : 32;
    static constexpr uint32_t sbytes = 128 / block;                     // scale bytes of 128 values
};

// Eight values, from the k-th on, into a staged row.  The order of a row inside a product
// is free, so it follows the lanes' loads of codes.  NVFP4: of 128 values lane t has the
// 32 from 32 t on (16 bytes), 8 for each of four steps.  MXFP4: of 32 (a block) lane t has
// 8 (4 bytes), in order.  MXFP8: of 32, 4 and the 4 that lie 16 further (4 bytes each).
template <int FMT>
__device__ __forceinline__ void stage8(char *row, uint32_t k, uint4 v, float f)
{
    const uint32_t x0 = half2_bits(bf16_lo(v.x) * f, bf16_hi(v.x) * f), x1 = half2_bits(bf16_lo(v.y) * f, bf16_hi(v.y) * f);
    const uint32_t x2 = half2_bits(bf16_lo(v.z) * f, bf16_hi(v.z) * f), x3 = half2_bits(bf16_lo(v.w) * f, bf16_hi(v.w) * f);
    if (FMT == MXQ_FMT_MXFP8) {
        char *to = row + ((k & ~31u) + (((k >> 2) & 3u) * 2u + ((k >> 4) & 1u)) * 4u) * 2u;
        *reinterpret_cast<uint2 *>(to) = make_uint2(x0, x1);
        *reinterpret_cast<uint2 *>(to + 16) = make_uint2(x2, x3);
    } else {
        const uint32_t at = FMT == MXQ_FMT_NVFP4 ? (k & ~127u) + ((k >> 3) & 3u) * 32u + ((k >> 5) & 3u) * 8u : k;
        *reinterpret_cast<uint4 *>(row + at * 2u) = make_uint4(x0, x1, x2, x3);
    }
}
__device__ __forceinline__ uint32_t largest8(uint4 v)
{
    return fold_halves(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(0u, v.x), v.y), v.z), v.w));
}

} // namespace

// A CTA brings one token into f16: its largest magnitude, then its values.
template <int FMT>
__global__ void __launch_bounds__(256)
linear_rows_kernel(const uint16_t *__restrict__ x, uint32_t K, uint32_t width, uint32_t *__restrict__ xh,
                   float *__restrict__ xf, uint32_t *__restrict__ status)
{
    __shared__ uint32_t part[8];
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();
    const uint16_t *src = x + (uint64_t)blockIdx.x * K;
    char *dst = reinterpret_cast<char *>(xh) + (uint64_t)blockIdx.x * width * 2u;
    uint32_t m = 0;
    for (uint32_t k = threadIdx.x * 8u; k < K; k += 2048u)
        m = max(m, largest8(__ldg(reinterpret_cast<const uint4 *>(src + k))));
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
    for (uint32_t k = threadIdx.x * 8u; k < width; k += 2048u)
        stage8<FMT>(dst, k, k < K ? __ldg(reinterpret_cast<const uint4 *>(src + k)) : make_uint4(0u, 0u, 0u, 0u), f);
}

template <int FMT, int NT, typename Out>
__global__ void __launch_bounds__(32 * kMostWarps, 1)
linear_kernel(const Args a)
{
    using F = Fmt<FMT>;
    extern __shared__ __align__(128) char smem[];
    __shared__ uint32_t xmax[kMostCap];         // CTA's own tokens: largest magnitudes
    __shared__ float xinv[kMostCap];            // inverse factors
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5, g8 = lane >> 2, t4 = lane & 3u;
    const uint32_t warps = blockDim.x >> 5, ring_bytes = a.slots * kSlot;
    char *ring = smem + warp * ring_bytes, *xs = smem + warps * ring_bytes;
    const uint32_t ring_s = smem_addr(ring);
    if (tid < kMostCap)
        xmax[tid] = 0u;
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();

    const uint32_t tok0 = blockIdx.y * a.cap, ntok = min(a.cap, a.T - tok0);
    float *part = reinterpret_cast<float *>(xs + a.cap * a.xstride);
    const uint32_t t0 = a.per * blockIdx.x + min(blockIdx.x, a.rest), t1 = t0 + a.per + (blockIdx.x < a.rest ? 1u : 0u);
    const uint32_t lg = a.kslog, ks = 1u << lg, teams = warps >> lg, team = warp >> lg, q = warp & (ks - 1u);
    const uint32_t c0 = (a.chunks * q) >> lg, c1 = (a.chunks * (q + 1u)) >> lg;

    const uint64_t once = once_policy();
    const uint32_t piece = lane & 7u;
    const uint32_t pdst = (lane >> 3) * F::pitch + (F::swap ? (piece * 16u) ^ ((lane >> 3 & 1u) * 64u) : piece * 16u);
    constexpr uint32_t spieces = F::groups;                 // scale pieces of a row of a chunk
    const uint32_t srow = lane / spieces, spiece = lane % spieces;
    uint32_t ptask = t0 + team, pch = c0, pslot = 0;
    const uint8_t *pcode[4], *pscale;
    auto locate = [&]() {       // rows past the last are read as the last: their sums are not stored
        const uint32_t r0 = ptask * 16u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            pcode[i] = a.codes + (uint64_t)min(r0 + (lane >> 3) + 4u * i, a.N - 1u) * a.row_bytes + piece * 16u;
        pscale = a.scales + (uint64_t)min(r0 + srow, a.N - 1u) * a.row_scales + spiece * F::sbytes;
    };
    auto issue = [&]() {
        if (ptask < t1) {
            const uint32_t dst = ring_s + pslot * kSlot + pdst, left = a.row_bytes - pch * kChunk;
            const bool in = piece * 16u < left;         // zeros behind the row's end
#pragma unroll
            for (int i = 0; i < 4; ++i)
                cp16_once(dst + 4 * i * F::pitch, pcode[i] + (in ? (uint64_t)pch * kChunk : 0ull), in, once);
            if (!a.direct && srow < 16u && spiece * F::group_bytes < left)
                cp_small<F::sbytes>(ring_s + pslot * kSlot + kScaleAt + srow * kScalePitch + spiece * F::sbytes,
                                    pscale + pch * (F::groups * F::sbytes));
            if (++pch == c1) {
                pch = c0;
                ptask += teams;
                if (ptask < t1)
                    locate();
            }
        }
        pslot = pslot + 1u == a.slots ? 0u : pslot + 1u;
        cp_commit();
    };

    // Token rows, and all but one slot of weights on their way.
    if (!a.x) {
        for (uint32_t i = tid; i < ntok * (a.width / 8u); i += blockDim.x) {
            const uint32_t r = fastdiv(i, a.rowdiv), p = i - r * (a.width / 8u);
            cp16(smem_addr(xs) + r * a.xstride + p * 16u,
                 reinterpret_cast<const char *>(a.xh) + ((uint64_t)(tok0 + r) * a.width + p * 8u) * 2u);
        }
        if (tid < ntok)
            xinv[tid] = __ldg(a.xf + tok0 + tid);
    }
    cp_commit();
    if (ptask < t1)
        locate();
    for (uint32_t i = 1; i < a.slots; ++i)
        issue();
    if (a.x) {
        const uint32_t pieces = ntok * (a.width / 8u);
        uint4 v[kOwnTurns];         // a thread's pieces
        uint32_t row[kOwnTurns], k[kOwnTurns];
#pragma unroll
        for (uint32_t n = 0; n < kOwnTurns; ++n)
            if (n * blockDim.x < pieces) {
                const uint32_t i = min(n * blockDim.x + tid, pieces - 1u);
                row[n] = fastdiv(i, a.rowdiv);
                k[n] = (i - row[n] * (a.width / 8u)) * 8u;
                const uint16_t *src = a.x + (uint64_t)(tok0 + row[n]) * a.K + k[n];
                v[n] = k[n] < a.K ? __ldg(reinterpret_cast<const uint4 *>(src)) : make_uint4(0u, 0u, 0u, 0u);
            }
        __syncthreads();            // xmax
#pragma unroll
        for (uint32_t n = 0; n < kOwnTurns; ++n)
            if (n * blockDim.x < pieces) {
                uint32_t m = largest8(v[n]);
                if (__all_sync(0xFFFFFFFFu, row[n] == __shfl_sync(0xFFFFFFFFu, row[n], 0))) {
                    m = __reduce_max_sync(0xFFFFFFFFu, m);
                    if (lane == 0)
                        atomicMax(&xmax[row[n]], m);
                } else
                    atomicMax(&xmax[row[n]], m);
            }
        __syncthreads();
#pragma unroll
        for (uint32_t n = 0; n < kOwnTurns; ++n)
            if (n * blockDim.x + tid < pieces)
                stage8<FMT>(xs + row[n] * a.xstride, k[n], v[n], row_factor(xmax[row[n]] << 16));
        if (tid < ntok) {
            const uint32_t m = xmax[tid] << 16;
            xinv[tid] = 1.0f / row_factor(m);
            if (m >= 0x7F800000u && blockIdx.x == 0)
                atomicOr(a.status, MXQ_DEV_NONFINITE_INPUT);
        }
    }
    if (a.slots == 2u)          // the tokens
        cp_wait<1>();
    else
        cp_wait<2>();
    __syncthreads();

    uint32_t slot = 0;
    uint32_t xoff[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i)        // columns without a token read the first one's row; their sums are not stored
        xoff[i] = (i * 8u + g8 < ntok ? i * 8u + g8 : 0u) * a.xstride + t4 * 16u;
    for (uint32_t task0 = t0; task0 < t1; task0 += teams) {
        const uint32_t task = task0 + team;
        float acc[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
            acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
        for (uint32_t ch = task < t1 ? c0 : c1; ch < c1; ++ch) {
            if (a.slots == 2u)
                cp_wait<0>();
            else
                cp_wait<1>();
            __syncwarp();
            issue();
            const char *cw = ring + slot * kSlot + g8 * F::pitch, *sb = ring + slot * kSlot + kScaleAt + g8 * kScalePitch;
            slot = slot + 1u == a.slots ? 0u : slot + 1u;
            uint32_t k = ch * F::chunk_k;
            const uint32_t groups = min(F::groups, (a.width - k) / 128u);
#pragma unroll 1
            for (uint32_t g = 0; g < groups; ++g, k += 128u) {
                uint32_t w0[2], w1[2];          // the scales of 128 values of both rows
                if (!a.direct) {
                    const char *p = sb + g * F::sbytes;
                    if (FMT == MXQ_FMT_NVFP4) {     // the lane's two
                        w0[0] = *reinterpret_cast<const uint16_t *>(p + t4 * 2u);
                        w1[0] = *reinterpret_cast<const uint16_t *>(p + t4 * 2u + 8 * kScalePitch);
                    } else {
                        w0[0] = lds32(p);
                        w1[0] = lds32(p + 8 * kScalePitch);
                    }
                } else {
                    const uint8_t *ds0 = a.scales + (uint64_t)min(task * 16u + g8, a.N - 1u) * a.row_scales;
                    const uint8_t *ds1 = a.scales + (uint64_t)min(task * 16u + g8 + 8u, a.N - 1u) * a.row_scales;
                    w0[0] = w0[1] = w1[0] = w1[1] = 0u;
                    const uint32_t n = min(a.K - k, 128u) / F::block;
                    for (uint32_t i = 0; i < n; ++i) {
                        w0[i >> 2] |= (uint32_t)__ldg(ds0 + k / F::block + i) << (8u * (i & 3u));
                        w1[i >> 2] |= (uint32_t)__ldg(ds1 + k / F::block + i) << (8u * (i & 3u));
                    }
                    if (FMT == MXQ_FMT_NVFP4) {
                        w0[0] = (t4 & 2u ? w0[1] : w0[0]) >> (t4 & 1u) * 16u;
                        w1[0] = (t4 & 2u ? w1[1] : w1[0]) >> (t4 & 1u) * 16u;
                    }
                }
                const char *xk = xs + k * 2u;
                if (FMT == MXQ_FMT_NVFP4) {
                    const char *p = cw + ((g ^ (g8 & 1u)) * 64u) + t4 * 16u;
                    const uint4 v0 = lds128(p), v1 = lds128(p + 8 * F::pitch);
                    const uint32_t q0[4] = {v0.x, v0.y, v0.z, v0.w}, q1[4] = {v1.x, v1.y, v1.z, v1.w};
                    const uint32_t s0 = e4m3x2_to_f16x2(w0[0]), s1 = e4m3x2_to_f16x2(w1[0]);
                    float run[NT][4];       // the sums of these 128 values
#pragma unroll
                    for (uint32_t u = 0; u < 4; ++u) {
                        uint32_t p0[4], p1[4];
                        e2m1x8_unpack(q0[u], p0);
                        e2m1x8_unpack(q1[u], p1);
                        const uint32_t e0 = u < 2 ? low2(s0) : high2(s0), e1 = u < 2 ? low2(s1) : high2(s1);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            p0[i] = hmul2_bits(p0[i], e0);
                            p1[i] = hmul2_bits(p1[i], e1);
                        }
#pragma unroll
                        for (int i = 0; i < NT; ++i) {
                            const uint4 b = lds128(xk + xoff[i] + u * 64u);
                            if (u == 0)
                                mma16816_first(run[i], p0[0], p1[0], p0[1], p1[1], b.x, b.y);
                            else
                                mma16816(run[i], p0[0], p1[0], p0[1], p1[1], b.x, b.y);
                            mma16816(run[i], p0[2], p1[2], p0[3], p1[3], b.z, b.w);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[i][j] += run[i][j];
                } else {
                    float d0[4], d1[4];
                    ue8m0x4(w0[0], d0);
                    ue8m0x4(w1[0], d1);
                    const char *q = cw + g * F::group_bytes + t4 * 4u;
#pragma unroll
                    for (uint32_t u = 0; u < 4; ++u) {           // a block of each row
                        uint32_t p0[4], p1[4];
                        if (F::fp4) {
                            e2m1x8_unpack(lds32(q + u * 16u), p0);
                            e2m1x8_unpack(lds32(q + u * 16u + 8 * F::pitch), p1);
                        } else {
                            e4m3x4_unpack(lds32(q + u * 32u), p0[0], p0[1]);
                            e4m3x4_unpack(lds32(q + u * 32u + 16), p0[2], p0[3]);
                            e4m3x4_unpack(lds32(q + u * 32u + 8 * F::pitch), p1[0], p1[1]);
                            e4m3x4_unpack(lds32(q + u * 32u + 8 * F::pitch + 16), p1[2], p1[3]);
                        }
#pragma unroll
                        for (int i = 0; i < NT; ++i) {
                            const uint4 b = lds128(xk + xoff[i] + u * 64u);
                            float c[4];
                            mma16816_first(c, p0[0], p1[0], p0[1], p1[1], b.x, b.y);
                            mma16816(c, p0[2], p1[2], p0[3], p1[3], b.z, b.w);
                            const float2 lo = __ffma2_rn(make_float2(c[0], c[1]), make_float2(d0[u], d0[u]),
                                                         make_float2(acc[i][0], acc[i][1]));
                            const float2 hi = __ffma2_rn(make_float2(c[2], c[3]), make_float2(d1[u], d1[u]),
                                                         make_float2(acc[i][2], acc[i][3]));
                            acc[i][0] = lo.x, acc[i][1] = lo.y, acc[i][2] = hi.x, acc[i][3] = hi.y;
                        }
                    }
                }
            }
        }
        if (ks > 1u) {          // the team's sums, in warp order
            float *mine = part + warp * (NT * 128u);
#pragma unroll
            for (int i = 0; i < NT; ++i)
                *reinterpret_cast<float4 *>(mine + (i * 32u + lane) * 4u) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
            named_barrier_sync(1 + (int)team, (int)(ks * 32u));
            if (q == 0)
                for (uint32_t w = 1; w < ks; ++w)
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const float4 v = *reinterpret_cast<const float4 *>(mine + w * (NT * 128u) + (i * 32u + lane) * 4u);
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
                        const float v = acc[i][j] * s2 * xinv[t];
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

constexpr uint32_t kSmemMax = 226 * 1024;       // dynamic

template <int FMT, int NT, typename Out>
cudaError_t go(const Args &a, dim3 grid, uint32_t warps, size_t smem, cudaStream_t s)
{
    const auto k = linear_kernel<FMT, NT, Out>;
    // always the largest, so that calls of other sizes from other threads set the same
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax);
    return e != cudaSuccess ? e : launch_dependent(k, grid, 32 * warps, smem, s, a);
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
    a.width = (a.K + 127) / 128 * 128;
    a.xstride = a.width * 2 + 64;       // 64 mod 128: rows of a fragment load fall on different banks
    a.direct = a.K % 128 != 0 || (reinterpret_cast<uintptr_t>(l.scales) % F::sbytes) != 0;
    a.rowdiv = make_fastdiv(a.width / 8);
    a.status = l.status;
    // As many tokens as fit beside 8 warps with two slots each, 32 at most, in groups of
    // about the same size.
    constexpr uint32_t sums = 512;          // bytes of a warp's sums for 8 tokens
    const uint32_t most = std::min<uint32_t>((kSmemMax - 8 * (2 * kSlot + 4 * sums)) / a.xstride, kMostCap);
    const uint32_t groups = (a.T + most - 1) / most;
    a.cap = (a.T + groups - 1) / groups;
    const uint32_t nt = a.cap <= 8 ? 1 : a.cap <= 16 ? 2 : 4, rows = a.cap * a.xstride;
    // One CTA an SM, of as many warps as fit with two slots each: the work on a chunk is a
    // chain of loads, conversions and products, and warps to switch to hide it.  With few
    // tasks several warps share one, so their number is a power of two.
    uint32_t warps = kMostWarps;
    while (warps > 8 && rows + warps * (2 * kSlot + nt * sums) > kSmemMax)
        warps -= a.tiles > (uint32_t)sms * 8 ? 2 : 8;
    a.slots = std::min((kSmemMax - rows - warps * nt * sums) / (warps * kSlot), kMostSlots);
    const uint32_t smem = rows + warps * (a.slots * kSlot + nt * sums);
    const uint32_t ctas = (uint32_t)std::min<uint64_t>((uint64_t)sms, a.tiles);
    a.per = a.tiles / ctas;
    a.rest = a.tiles % ctas;
    a.kslog = 0;
    while (a.kslog < 3 && warps % (2u << a.kslog) == 0 && (2u << a.kslog) <= a.chunks &&
           ((uint64_t)a.tiles * 2 << a.kslog) <= (uint64_t)ctas * warps)
        ++a.kslog;
    // A CTA's own work on the tokens costs less than another kernel before it where a
    // thread can hold its share.
    a.x = a.cap * (a.width / 8) <= kOwnTurns * 32 * warps ? l.x : nullptr;
    cudaError_t e = cudaSuccess;
    if (!a.x)
        e = launch_dependent(linear_rows_kernel<FMT>, dim3(a.T), 256, 0, s, l.x, a.K, a.width, l.xh, l.xf, l.status);
    if (e != cudaSuccess)
        return e;
    const dim3 grid(ctas, groups);
    if (out_f32)
        return nt == 1   ? go<FMT, 1, float>(a, grid, warps, smem, s)
               : nt == 2 ? go<FMT, 2, float>(a, grid, warps, smem, s)
                         : go<FMT, 4, float>(a, grid, warps, smem, s);
    return nt == 1   ? go<FMT, 1, __nv_bfloat16>(a, grid, warps, smem, s)
           : nt == 2 ? go<FMT, 2, __nv_bfloat16>(a, grid, warps, smem, s)
                     : go<FMT, 4, __nv_bfloat16>(a, grid, warps, smem, s);
}

} // namespace

size_t linear_rows_bytes(int64_t T, int64_t K) { return (size_t)T * (size_t)((K + 127) / 128 * 128) * 2; }
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
