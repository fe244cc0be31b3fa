// moe.cu -- a whole mixture-of-experts layer for a few tokens over
// block-scaled expert weights (sm_100a).
//
//   y[t] = sum_j w[t,j] D_e (silu(G_e x_t) * (U_e x_t)),  e = ids[t,j]
//
// with G_e, U_e the two halves of the fused gate_up slab (rows [0, I) and
// [I, 2I)), D_e the down slab, each dequantized on the fly from NVFP4, MXFP4,
// MXFP8 or block-FP8 codes.  Few tokens share an expert, so the work is the
// read of each chosen expert's codes and scales: HBM is the bound and the
// arithmetic only has to keep out of its way.
//
// Three launches, each allowed to start while the one before drains
// (programmatic dependent launch; the second fetches its first weights before
// it waits):
//   moe_kernel<FMT, true>   h[a] = silu(G x) * (U x)        fp32 [A, I]
//   moe_kernel<FMT, false>  z[a] = w[a] D h[a]              fp32 [A, H]
//   moe_combine_kernel      y[t] = sum_j z[t k + j]         fixed order
// a = t k + j numbers the assignments.  Each z row is written by one warp and
// summed in the order of j, so repeated calls give the same bits.
//
// moe_kernel.  One CTA of 16 warps per SM.  Every CTA builds the list of
// chosen experts itself (at most 2048 assignments).  An expert's assignments
// are cut into groups of at most 8; a task is 16 weight rows (gate_up: 8 gate
// rows and the same 8 up rows, so the activation is local to a thread) of one
// group, over the whole length K; a CTA takes a contiguous run of tasks, so
// it reads contiguous rows and needs the activations of few groups.
//
// Weights.  A warp streams its tasks through its own ring of chunks (16 rows
// of 128 bytes of codes and their scales) in shared memory with cp.async, so
// no warp waits for another one's data; with few tasks 2, 4, ... warps split K
// and add their sums in a fixed order.  The 16-byte pieces of a row are
// permuted (xor) so that the fragment loads have no bank conflicts.
//
// Product.  mma.sync m16n8k16 with f16 operands and fp32 sums: 16 weight rows
// by 8 assignments.  Few columns are filled, and the tensor pipe is idle most
// of the time, so the fifth-generation instructions, which take their weights
// from shared memory in the packed formats (or decoded and written back
// there), would only add traffic.  E2M1 and E4M3 values are exact in f16, and
// so is E2M1 x E4M3 scale (6 significant bits, 2^-10 to 2688): NVFP4 codes are
// multiplied by their block scale in f16, exactly.  UE8M0 and fp32 scales
// multiply the fp32 sum of their block instead.
//
// Activations.  Each row is held in f16 times the power of two that brings
// its largest magnitude into [2^14, 2^15): for bf16 tokens that is exact for
// every element above 2^-31 of the largest, and below it off by at most 2^-39
// of the largest.  The fp32 h rows are rounded to f16's 11 bits (relative
// 2^-11 a value, an eighth of the bf16 output's own rounding).
#include "mxq_device.cuh"
#include "mxq_internal.h"
#include "mxq.h"

namespace mxq {

namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kCodeBytes = 16 * 128;             // codes of one chunk
constexpr int kSlotBytes = kCodeBytes + 256;     // and its scales
constexpr int kGroup = 8;                        // assignments of a group (columns of the product)

struct MoeArgs {
    const uint16_t *x;          // gate_up: bf16 tokens [T, K]
    const float *hin;           // down: fp32 rows [A, K]
    const int32_t *ids;         // [A]
    const float *w;             // down: [A]
    const uint8_t *codes;       // [E, rows, K * bits / 8]
    const void *scales;
    const float *s2;            // NVFP4: [E]
    float *out;                 // gate_up: h [A, I]; down: z [A, H]
    uint32_t *status;
    uint64_t expert_bytes;      // codes of one expert
    uint64_t expert_scales;     // scales of one expert (bytes)
    uint32_t row_bytes;         // codes of one row
    uint32_t row_scales;        // scales of one row (bytes); block-FP8: of one row of blocks
    uint32_t A, topk, E, K;
    uint32_t nrows;             // rows of an output: I or H
    uint32_t tiles;             // tasks of a group
    uint32_t chunks;            // chunks of a row
    uint32_t cap;               // activation rows the stage holds
    uint32_t xstride;           // bytes of a staged row
    FastDiv tilesdiv, topkdiv;
};

template <int FMT>
struct Fmt {
    static constexpr bool fp4 = FMT == MXQ_FMT_NVFP4 || FMT == MXQ_FMT_MXFP4;
    static constexpr int chunk_k = fp4 ? 256 : 128;                       // values of a row in a chunk
    // scale bytes of a row in a chunk
    static constexpr int sbytes = FMT == MXQ_FMT_NVFP4 ? 16 : FMT == MXQ_FMT_MXFP4 ? 8 : 4;
    // 4-bit fragments take one word of each of 8 rows at one piece, 8-bit
    // ones two words of each of 4 rows at two pieces
    static __device__ __forceinline__ uint32_t swz(uint32_t row) { return fp4 ? (row & 7u) : (row & 3u) << 1; }
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_small(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t lds32(const char *p) { return *reinterpret_cast<const uint32_t *>(p); }
__device__ __forceinline__ uint2 lds64(const char *p) { return *reinterpret_cast<const uint2 *>(p); }
__device__ __forceinline__ uint4 lds128(const char *p) { return *reinterpret_cast<const uint4 *>(p); }

// c += A B: A 16 rows x 16 k (f16), B 16 k x 8 columns (f16).
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// UE8M0 byte -> fp32 2^(b - 127); 255 is NaN.
__device__ __forceinline__ float ue8m0(uint32_t b)
{
    const uint32_t bits = b ? b << 23 : 0x00400000u;
    return __uint_as_float(b == 255u ? 0x7FC00000u : bits);
}

// The chosen experts.  list: assignments sorted by expert; group g holds
// list[start[g] .. start[g + 1]) of expert expert[g], at most kGroup of them.
struct Route {
    uint16_t *list, *start, *expert;
    uint32_t groups;
};

// Up to 32 assignments: one warp, by matching ids.
__device__ __forceinline__ uint32_t route_warp(const MoeArgs &a, const Route &r, uint32_t lane)
{
    int id = lane < a.A ? a.ids[lane] : -1;
    if (id >= (int)a.E) {
        atomicOr(a.status, MXQ_DEV_INVALID_EXPERT);
        id = -1;
    }
    const uint32_t peers = __match_any_sync(0xFFFFFFFFu, id), below = (1u << lane) - 1u;
    const uint32_t n = __popc(peers), rank = __popc(peers & below);
    const bool lead = id >= 0 && rank == 0;
    // exclusive sums over the leaders below: groups (high half), assignments
    uint32_t v = lead ? (((n + kGroup - 1) / kGroup) << 16) | n : 0u;
    const uint32_t own = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= (uint32_t)o)
            v += u;
    }
    const uint32_t total = __shfl_sync(0xFFFFFFFFu, v, 31);
    const uint32_t base = __shfl_sync(0xFFFFFFFFu, v - own, __ffs(peers) - 1);
    if (id >= 0) {
        r.list[(base & 0xFFFFu) + rank] = (uint16_t)lane;
        if (rank % kGroup == 0) {
            r.start[(base >> 16) + rank / kGroup] = (uint16_t)((base & 0xFFFFu) + rank);
            r.expert[(base >> 16) + rank / kGroup] = (uint16_t)id;
        }
    }
    if (lane == 0)
        r.start[total >> 16] = (uint16_t)(total & 0xFFFFu);
    return total >> 16;
}

// More: counts per expert in shared memory (E words at `cnt`), a scan, and a
// scatter by the first warp, 32 assignments at a time in their order: an
// expert's groups have to be the same in every CTA.  The list is complete at
// the next barrier of the CTA; groups and experts are at the return.
__device__ __forceinline__ uint32_t route_block(const MoeArgs &a, const Route &r, uint32_t *cnt, uint32_t *wsum)
{
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    for (uint32_t e = tid; e < a.E; e += kThreads)
        cnt[e] = 0u;
    __syncthreads();
    for (uint32_t i = tid; i < a.A; i += kThreads) {
        const int id = a.ids[i];
        if (id >= (int)a.E)
            atomicOr(a.status, MXQ_DEV_INVALID_EXPERT);
        else if (id >= 0)
            atomicAdd(&cnt[id], 1u);
    }
    __syncthreads();
    const uint32_t per = (a.E + kThreads - 1) / kThreads, e0 = min(tid * per, a.E), e1 = min(e0 + per, a.E);
    uint32_t own = 0;
    for (uint32_t e = e0; e < e1; ++e)
        own += (((cnt[e] + kGroup - 1) / kGroup) << 16) | cnt[e];
    uint32_t v = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= (uint32_t)o)
            v += u;
    }
    if (lane == 31u)
        wsum[warp] = v;
    __syncthreads();
    uint32_t total = 0;
    for (uint32_t i = 0; i < kWarps; ++i) {
        if (i < warp)
            v += wsum[i];
        total += wsum[i];
    }
    v -= own;
    for (uint32_t e = e0; e < e1; ++e) {
        const uint32_t n = cnt[e];
        cnt[e] = v & 0xFFFFu;
        for (uint32_t i = 0; i < n; i += kGroup) {
            r.start[v >> 16] = (uint16_t)(v & 0xFFFFu);
            r.expert[v >> 16] = (uint16_t)e;
            v += (1u << 16) + min(n - i, (uint32_t)kGroup);
        }
    }
    if (tid == 0)
        r.start[total >> 16] = (uint16_t)(total & 0xFFFFu);
    __syncthreads();
    if (warp == 0)
        for (uint32_t i = lane; i < ((a.A + 31u) & ~31u); i += 32u) {
            int id = i < a.A ? a.ids[i] : -1;
            if (id >= (int)a.E)
                id = -1;
            const uint32_t peers = __match_any_sync(0xFFFFFFFFu, id), rank = __popc(peers & ((1u << lane) - 1u));
            uint32_t at = 0;
            if (id >= 0) {
                at = cnt[id];
                r.list[at + rank] = (uint16_t)i;
            }
            __syncwarp();
            if (id >= 0 && rank == 0)
                cnt[id] = at + __popc(peers);
            __syncwarp();
        }
    return total >> 16;
}

// Power of two that brings a magnitude of these fp32 bits into [2^14, 2^15),
// as the bits of its factor; 1 for zero, Inf and NaN.  The exponent is kept
// within 126, so tiny rows land lower.
__device__ __forceinline__ float row_factor(uint32_t amax_bits)
{
    const int e = (int)(amax_bits >> 23) - 127;
    if (amax_bits == 0u || e == 128)
        return 1.0f;
    return __uint_as_float((uint32_t)(127 + min(max(14 - e, -126), 126)) << 23);
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// One warp: row `a` of the activations -> f16 at `dst`, its inverse factor
// returned.
template <bool GATE_UP>
__device__ __forceinline__ float stage_row(const MoeArgs &g, uint32_t a, char *dst, uint32_t lane)
{
    uint32_t m = 0;
    if (GATE_UP) {
        const uint16_t *src = g.x + (uint64_t)fastdiv(a, g.topkdiv) * g.K;
        for (uint32_t k = lane * 8u; k < g.K; k += 256u) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src + k));
            uint32_t q = absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(0u, v.x), v.y), v.z), v.w);
            m = max(m, fold_halves(q));
        }
        m = __reduce_max_sync(0xFFFFFFFFu, m) << 16;
        if (m >= 0x7F800000u && lane == 0)
            atomicOr(g.status, MXQ_DEV_NONFINITE_INPUT);
        const float f = row_factor(m);
        for (uint32_t k = lane * 8u; k < g.K; k += 256u) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src + k));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                h[i] = half2_bits(bf16_lo(w[i]) * f, bf16_hi(w[i]) * f);
            *reinterpret_cast<uint4 *>(dst + k * 2u) = make_uint4(h[0], h[1], h[2], h[3]);
        }
        return 1.0f / f;
    }
    const float *src = g.hin + (uint64_t)a * g.K;
    for (uint32_t k = lane * 4u; k < g.K; k += 128u) {
        const float4 v = *reinterpret_cast<const float4 *>(src + k);
        m = max(max(m, max(__float_as_uint(fabsf(v.x)), __float_as_uint(fabsf(v.y)))),
                max(__float_as_uint(fabsf(v.z)), __float_as_uint(fabsf(v.w))));
    }
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    const float f = row_factor(m >= 0x7F800000u ? 0u : m);
    for (uint32_t k = lane * 4u; k < g.K; k += 128u) {
        const float4 v = *reinterpret_cast<const float4 *>(src + k);
        *reinterpret_cast<uint2 *>(dst + k * 2u) =
            make_uint2(half2_bits(v.x * f, v.y * f), half2_bits(v.z * f, v.w * f));
    }
    return 1.0f / f;
}

// A warp's walk over its (task, chunk) pairs.
struct Walk {
    uint32_t task, ch;
    const uint8_t *code;        // this lane's first piece of the task's first row
    const char *scale;          // this lane's scales
};

} // namespace

template <int FMT, bool GATE_UP, int D>
__global__ void __launch_bounds__(kThreads, 1)
moe_kernel(const MoeArgs a)
{
    using F = Fmt<FMT>;
    extern __shared__ __align__(128) char smem[];
    __shared__ uint32_t wsum[kWarps];
    __shared__ uint32_t groups_s;
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5, g8 = lane >> 2, t4 = lane & 3u;
    // shared memory: rings, activation rows, row factors, lists, partial sums
    char *ring = smem + warp * (D * kSlotBytes);
    char *xs = smem + kWarps * D * kSlotBytes;
    float *xf = reinterpret_cast<float *>(xs + a.cap * a.xstride);
    float *part = xf + ((a.cap + 3u) & ~3u);
    Route r;
    r.list = reinterpret_cast<uint16_t *>(part + kWarps * 128);
    r.start = r.list + a.A;
    r.expert = r.start + a.A + 1;
    if (a.A <= 32u) {
        if (warp == 0) {
            const uint32_t n = route_warp(a, r, lane);
            if (lane == 0)
                groups_s = n;
        }
        __syncthreads();
        r.groups = groups_s;
    } else
        r.groups = route_block(a, r, reinterpret_cast<uint32_t *>(xs), wsum);
    // this CTA's run of tasks
    const uint32_t ntask = r.groups * a.tiles;
    const uint32_t t0 = (uint32_t)((uint64_t)ntask * blockIdx.x / gridDim.x);
    const uint32_t t1 = (uint32_t)((uint64_t)ntask * (blockIdx.x + 1) / gridDim.x);
    // warps that share a task: doubled while every warp of the grid still gets
    // at most one and each has a chunk
    uint32_t ks = 1;
    while (ks * 2u <= kWarps && ks * 2u <= a.chunks && (uint64_t)ntask * ks * 2u <= (uint64_t)gridDim.x * kWarps)
        ks *= 2u;
    const uint32_t teams = kWarps / ks, team = warp / ks, q = warp - team * ks;
    const uint32_t c0 = a.chunks * q / ks, c1 = a.chunks * (q + 1) / ks;

    const uint32_t half = GATE_UP ? a.nrows : 8u;    // distance of the second 8 rows from the first
    const uint32_t tile_rows = GATE_UP ? 8u : 16u;
    const uint32_t piece = lane & 7u;
    const uint32_t ring_s = smem_addr(ring);
    Walk p;
    p.task = t0 + team;
    p.ch = c0;
    auto locate = [&]() {
        const uint32_t grp = fastdiv(p.task, a.tilesdiv), tile = p.task - grp * a.tiles, e = r.expert[grp];
        const uint32_t r0 = tile * tile_rows;
        p.code = a.codes + e * a.expert_bytes + (uint64_t)(r0 + (lane >> 3)) * a.row_bytes + piece * 16u;
        const char *se = static_cast<const char *>(a.scales) + e * a.expert_scales;
        if (FMT == MXQ_FMT_FP8_BLOCK)      // lanes 0, 1: the block rows of the two halves
            p.scale = se + (uint64_t)((r0 + (lane & 1u) * half) >> 7) * a.row_scales;
        else {
            // fp4: two lanes a row, half of its bytes each; MXFP8: one lane a row
            const uint32_t row = F::fp4 ? lane >> 1 : lane & 15u;
            p.scale = se + (uint64_t)(r0 + (row & 7u) + (row >> 3) * half) * a.row_scales +
                      (F::fp4 ? (lane & 1u) * (F::sbytes / 2) : 0u);
        }
    };
    auto issue = [&](uint32_t slot) {
        if (p.task < t1) {
            const uint32_t dst = ring_s + slot * kSlotBytes, off = p.ch * 128u, row = lane >> 3;
            if (off + piece * 16u < a.row_bytes) {
                const uint8_t *s = p.code + off;
                const uint64_t r4 = 4ull * a.row_bytes, hb = (uint64_t)half * a.row_bytes;
                // row + 4 i: its swizzle, too, follows from the row
                cp16(dst + row * 128u + ((piece ^ F::swz(row)) << 4), s);
                cp16(dst + (row + 4u) * 128u + ((piece ^ F::swz(row + 4u)) << 4), s + r4);
                cp16(dst + (row + 8u) * 128u + ((piece ^ F::swz(row)) << 4), s + hb);
                cp16(dst + (row + 12u) * 128u + ((piece ^ F::swz(row + 4u)) << 4), s + hb + r4);
            }
            const uint32_t sd = dst + kCodeBytes;
            if (FMT == MXQ_FMT_NVFP4) {
                if (p.ch * 16u + (lane & 1u) * 8u < a.row_scales)
                    cp_small<8>(sd + lane * 8u, p.scale + p.ch * 16u);
            } else if (FMT == MXQ_FMT_MXFP4) {
                if (p.ch * 8u + (lane & 1u) * 4u < a.row_scales)
                    cp_small<4>(sd + lane * 4u, p.scale + p.ch * 8u);
            } else if (FMT == MXQ_FMT_MXFP8) {
                if (lane < 16u)
                    cp_small<4>(sd + lane * 4u, p.scale + p.ch * 4u);
            } else if (lane < 2u)
                cp_small<4>(sd + lane * 4u, p.scale + p.ch * 4u);
            if (++p.ch == c1) {
                p.ch = c0;
                p.task += teams;
                if (p.task < t1)
                    locate();
            }
        }
        cp_commit();
    };
    if (p.task < t1)
        locate();
#pragma unroll
    for (int i = 0; i < D - 1; ++i)
        issue(i);
    if (!GATE_UP)
        cudaGridDependencySynchronize();     // h is written by the launch before
    cudaTriggerProgrammaticLaunchCompletion();

    uint32_t slot = 0, pos = t0, task = t0 + team;
    while (pos < t1) {
        // activations of as many groups as the stage holds
        const uint32_t g0 = fastdiv(pos, a.tilesdiv), row0 = r.start[g0];
        uint32_t gl = g0 + 1;
        const uint32_t gend = fastdiv(t1 - 1u, a.tilesdiv) + 1u;
        while (gl < gend && (uint32_t)r.start[gl + 1] - row0 <= a.cap)
            ++gl;
        const uint32_t end = min(t1, gl * a.tiles), nr = (uint32_t)r.start[gl] - row0;
        __syncthreads();
        for (uint32_t i = warp; i < nr; i += kWarps) {
            const float f = stage_row<GATE_UP>(a, r.list[row0 + i], xs + i * a.xstride, lane);
            if (lane == 0)
                xf[i] = f;
        }
        __syncthreads();
        for (; task < end; task += teams) {
            const uint32_t grp = fastdiv(task, a.tilesdiv), tile = task - grp * a.tiles;
            const uint32_t first = r.start[grp], cnt = r.start[grp + 1] - first;
            const bool col = g8 < cnt;
            const char *xrow = xs + (first - row0 + (col ? g8 : 0u)) * a.xstride + t4 * 16u;
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            for (uint32_t ch = c0; ch < c1; ++ch) {
                cp_wait<D - 2>();
                __syncwarp();
                issue(slot == 0 ? D - 1 : slot - 1);     // the slot read in the step before
                const char *base = ring + slot * kSlotBytes, *sb = base + kCodeBytes;
                slot = slot == D - 1 ? 0 : slot + 1;
                const char *xk = xrow + ch * (F::chunk_k * 2u);
                const uint32_t nk = min((uint32_t)F::chunk_k, a.K - ch * F::chunk_k);
                if (FMT == MXQ_FMT_NVFP4) {
                    const uint4 s0 = lds128(sb + g8 * 16u), s1 = lds128(sb + 128u + g8 * 16u);
                    const uint32_t w0[4] = {s0.x, s0.y, s0.z, s0.w}, w1[4] = {s1.x, s1.y, s1.z, s1.w};
#pragma unroll
                    for (uint32_t hk = 0; hk < 2; ++hk) {
                        if (hk * 128u >= nk)
                            break;
#pragma unroll
                        for (uint32_t u2 = 0; u2 < 4; ++u2) {
                            const uint32_t u = hk * 4u + u2, sel = ((u & 1u) * 2u + (t4 >> 1)) * 0x11u;
                            const uint32_t d0 = e4m3x2_to_f16x2(__byte_perm(w0[u >> 1], 0u, sel));
                            const uint32_t d1 = e4m3x2_to_f16x2(__byte_perm(w1[u >> 1], 0u, sel));
                            const char *at = base + g8 * 128u + ((u ^ g8) << 4) + t4 * 4u;
                            uint32_t p0[4], p1[4];
                            e2m1x8_to_f16x2(lds32(at), p0);
                            e2m1x8_to_f16x2(lds32(at + 1024u), p1);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                p0[i] = hmul2_bits(p0[i], d0);
                                p1[i] = hmul2_bits(p1[i], d1);
                            }
                            uint4 b = lds128(xk + u * 64u);
                            if (!col)
                                b = make_uint4(0u, 0u, 0u, 0u);
                            mma16816(acc, p0[0], p1[0], p0[1], p1[1], b.x, b.y);
                            mma16816(acc, p0[2], p1[2], p0[3], p1[3], b.z, b.w);
                        }
                    }
                } else if (FMT == MXQ_FMT_MXFP4) {
                    const uint2 s0 = lds64(sb + g8 * 8u), s1 = lds64(sb + 64u + g8 * 8u);
                    const uint32_t w0[2] = {s0.x, s0.y}, w1[2] = {s1.x, s1.y};
#pragma unroll
                    for (uint32_t hk = 0; hk < 2; ++hk) {
                        if (hk * 128u >= nk)
                            break;
#pragma unroll
                        for (uint32_t u2 = 0; u2 < 4; ++u2) {
                            const uint32_t u = hk * 4u + u2;
                            const char *at = base + g8 * 128u + ((u ^ g8) << 4) + t4 * 4u;
                            uint32_t p0[4], p1[4];
                            e2m1x8_to_f16x2(lds32(at), p0);
                            e2m1x8_to_f16x2(lds32(at + 1024u), p1);
                            uint4 b = lds128(xk + u * 64u);
                            if (!col)
                                b = make_uint4(0u, 0u, 0u, 0u);
                            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                            mma16816(c, p0[0], p1[0], p0[1], p1[1], b.x, b.y);
                            mma16816(c, p0[2], p1[2], p0[3], p1[3], b.z, b.w);
                            const float d0 = ue8m0((w0[hk] >> (8u * u2)) & 255u);
                            const float d1 = ue8m0((w1[hk] >> (8u * u2)) & 255u);
                            acc[0] = fmaf(c[0], d0, acc[0]);
                            acc[1] = fmaf(c[1], d0, acc[1]);
                            acc[2] = fmaf(c[2], d1, acc[2]);
                            acc[3] = fmaf(c[3], d1, acc[3]);
                        }
                    }
                } else {
                    const uint32_t w0 = lds32(sb + (FMT == MXQ_FMT_MXFP8 ? g8 * 4u : 0u));
                    const uint32_t w1 = lds32(sb + (FMT == MXQ_FMT_MXFP8 ? 32u + g8 * 4u : 4u));
                    float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (uint32_t u = 0; u < 4; ++u) {
                        const char *at = base + g8 * 128u + (((2u * u + (t4 >> 1)) ^ F::swz(g8)) << 4) + (t4 & 1u) * 8u;
                        const uint2 v0 = lds64(at), v1 = lds64(at + 1024u);
                        uint4 b = lds128(xk + u * 64u);
                        if (!col)
                            b = make_uint4(0u, 0u, 0u, 0u);
                        mma16816(c, e4m3x2_to_f16x2(v0.x), e4m3x2_to_f16x2(v1.x), e4m3x2_to_f16x2(v0.x >> 16),
                                 e4m3x2_to_f16x2(v1.x >> 16), b.x, b.y);
                        mma16816(c, e4m3x2_to_f16x2(v0.y), e4m3x2_to_f16x2(v1.y), e4m3x2_to_f16x2(v0.y >> 16),
                                 e4m3x2_to_f16x2(v1.y >> 16), b.z, b.w);
                        if (FMT == MXQ_FMT_MXFP8) {
                            const float d0 = ue8m0((w0 >> (8u * u)) & 255u), d1 = ue8m0((w1 >> (8u * u)) & 255u);
                            acc[0] = fmaf(c[0], d0, acc[0]);
                            acc[1] = fmaf(c[1], d0, acc[1]);
                            acc[2] = fmaf(c[2], d1, acc[2]);
                            acc[3] = fmaf(c[3], d1, acc[3]);
                            c[0] = c[1] = c[2] = c[3] = 0.0f;
                        }
                    }
                    if (FMT == MXQ_FMT_FP8_BLOCK) {
                        const float d0 = __uint_as_float(w0), d1 = __uint_as_float(w1);
                        acc[0] = fmaf(c[0], d0, acc[0]);
                        acc[1] = fmaf(c[1], d0, acc[1]);
                        acc[2] = fmaf(c[2], d1, acc[2]);
                        acc[3] = fmaf(c[3], d1, acc[3]);
                    }
                }
            }
            if (ks > 1) {       // the team's partial sums, in warp order
                *reinterpret_cast<float4 *>(part + warp * 128u + lane * 4u) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                named_barrier_sync(1 + (int)team, (int)(ks * 32u));
                if (q == 0)
                    for (uint32_t i = 1; i < ks; ++i) {
                        const float4 v = *reinterpret_cast<const float4 *>(part + (warp + i) * 128u + lane * 4u);
                        acc[0] += v.x;
                        acc[1] += v.y;
                        acc[2] += v.z;
                        acc[3] += v.w;
                    }
                named_barrier_sync(1 + (int)team, (int)(ks * 32u));
            }
            if (q == 0) {
                const float s2 = FMT == MXQ_FMT_NVFP4 ? a.s2[r.expert[grp]] : 1.0f;
#pragma unroll
                for (uint32_t c = 0; c < 2; ++c) {
                    const uint32_t n = t4 * 2u + c;
                    if (n < cnt) {
                        const uint32_t as = r.list[first + n];
                        const float f = xf[first - row0 + n];
                        const float lo = acc[c] * s2 * f, hi = acc[2 + c] * s2 * f;
                        if (GATE_UP)
                            a.out[(uint64_t)as * a.nrows + tile * 8u + g8] = lo / (1.0f + expf(-lo)) * hi;
                        else {
                            const float w = a.w[as];
                            float *o = a.out + (uint64_t)as * a.nrows + tile * 16u + g8;
                            o[0] = lo * w;
                            o[8] = hi * w;
                        }
                    }
                }
            }
        }
        pos = end;
    }
    cp_wait<0>();
}

// y[t] = sum over the token's experts of z, in their order; 4 columns a thread.
__global__ void __launch_bounds__(128)
moe_combine_kernel(const float *__restrict__ z, const int32_t *__restrict__ ids, uint32_t T, uint32_t topk,
                   uint32_t E, uint32_t H, uint16_t *__restrict__ y)
{
    cudaGridDependencySynchronize();
    const uint32_t h = (blockIdx.x * 128u + threadIdx.x) * 4u, t = blockIdx.y;
    if (h >= H)
        return;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (uint32_t j = 0; j < topk; ++j) {
        const int id = ids[t * topk + j];
        if (id < 0 || id >= (int)E)
            continue;
        const float4 v = *reinterpret_cast<const float4 *>(z + (uint64_t)(t * topk + j) * H + h);
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    }
    const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
    *reinterpret_cast<uint2 *>(y + (uint64_t)t * H + h) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
}

namespace {

template <typename... P, typename... Q>
cudaError_t launch(void (*k)(P...), dim3 grid, unsigned block, size_t smem, bool dependent, cudaStream_t s, Q... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = dependent ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k, args...);
}

constexpr size_t kSmemMax = 227 * 1024 - 256;     // less the static words of the kernel

template <int FMT, bool GATE_UP, int D>
cudaError_t run(MoeArgs a, size_t smem, int ctas, cudaStream_t s)
{
    const auto k = moe_kernel<FMT, GATE_UP, D>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess)
        return e;
    return launch(k, dim3((unsigned)ctas), kThreads, smem, !GATE_UP, s, a);
}

template <int FMT, bool GATE_UP>
cudaError_t moe_gemm(MoeArgs a, int ctas, cudaStream_t s)
{
    a.row_bytes = Fmt<FMT>::fp4 ? a.K / 2 : a.K;
    a.row_scales = FMT == MXQ_FMT_NVFP4 ? a.K / 16 : FMT == MXQ_FMT_FP8_BLOCK ? a.K / 128 * 4 : a.K / 32;
    const uint64_t rows = GATE_UP ? 2ull * a.nrows : a.nrows;
    a.expert_bytes = rows * a.row_bytes;
    a.expert_scales = (FMT == MXQ_FMT_FP8_BLOCK ? rows / 128 : rows) * a.row_scales;
    a.tiles = a.nrows / (GATE_UP ? 8 : 16);
    a.tilesdiv = make_fastdiv(a.tiles);
    a.topkdiv = make_fastdiv(a.topk);
    a.chunks = (a.K + Fmt<FMT>::chunk_k - 1) / Fmt<FMT>::chunk_k;
    a.xstride = a.K * 2 + 64;       // 64 mod 128: the rows of a fragment load fall on different banks
    const size_t lists = (3 * (size_t)a.A + 2) * 2 + 64;
    const size_t fixed = kWarps * 128 * 4 + lists;
    // ring of 4 chunks a warp where 8 activation rows fit beside it, else 2
    const int depth = kWarps * 4 * kSlotBytes + fixed + 8 * (a.xstride + 4) + 16 <= kSmemMax ? 4 : 2;
    const size_t ring = (size_t)kWarps * depth * kSlotBytes;
    uint32_t cap = (uint32_t)((kSmemMax - ring - fixed - 16) / (a.xstride + 4));
    a.cap = cap > 64 ? 64 : cap;    // at least 16 KB in all: the expert counts lie there first
    const size_t smem = ring + fixed + a.cap * (size_t)a.xstride + (((size_t)a.cap + 3) & ~3ull) * 4;
    return depth == 4 ? run<FMT, GATE_UP, 4>(a, smem, ctas, s) : run<FMT, GATE_UP, 2>(a, smem, ctas, s);
}

template <int FMT>
cudaError_t moe_all(const MoeLayer &m, int sms, cudaStream_t s)
{
    MoeArgs a = {};
    a.x = m.x;
    a.hin = m.h;
    a.ids = m.ids;
    a.w = m.weights;
    a.status = m.status;
    a.A = (uint32_t)(m.T * m.topk);
    a.topk = (uint32_t)m.topk;
    a.E = (uint32_t)m.experts;
    a.codes = m.gu_codes;
    a.scales = m.gu_scales;
    a.s2 = m.gu_s2;
    a.out = m.h;
    a.K = (uint32_t)m.hidden;
    a.nrows = (uint32_t)m.inter;
    cudaError_t e = moe_gemm<FMT, true>(a, sms, s);
    if (e != cudaSuccess)
        return e;
    a.codes = m.dn_codes;
    a.scales = m.dn_scales;
    a.s2 = m.dn_s2;
    a.out = m.z;
    a.K = (uint32_t)m.inter;
    a.nrows = (uint32_t)m.hidden;
    e = moe_gemm<FMT, false>(a, sms, s);
    if (e != cudaSuccess)
        return e;
    return launch(moe_combine_kernel, dim3((unsigned)((m.hidden + 511) / 512), (unsigned)m.T), 128, 0, true, s,
                  (const float *)m.z, m.ids, (uint32_t)m.T, a.topk, a.E, (uint32_t)m.hidden, m.y);
}

} // namespace

cudaError_t launch_moe(const MoeLayer &m, int fmt, cudaStream_t s)
{
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return e;
    switch (fmt) {
    case MXQ_FMT_NVFP4: return moe_all<MXQ_FMT_NVFP4>(m, sms, s);
    case MXQ_FMT_MXFP4: return moe_all<MXQ_FMT_MXFP4>(m, sms, s);
    case MXQ_FMT_MXFP8: return moe_all<MXQ_FMT_MXFP8>(m, sms, s);
    default: return moe_all<MXQ_FMT_FP8_BLOCK>(m, sms, s);
    }
}

} // namespace mxq
