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
// Up to three launches, each allowed to start while the one before drains
// (programmatic dependent launch; the second fetches its first weights before
// it waits for h, which the first's own wait at its start allows):
//   moe_kernel<FMT, true>   h[a] = silu(G x) * (U x)        fp32 [A, I]
//   moe_kernel<FMT, false>  z[a] = w[a] D h[a]              fp32 [A, H]
//   moe_combine_kernel      y[t] = sum_j z[t k + j]         fixed order
// (the second adds up y itself, two launches in all, where there is little to do).
// a = t k + j numbers the assignments.  Each z row is written by one warp and
// summed in the order of j, so repeated calls give the same bits.
//
// moe_kernel.  One CTA of 16 warps (8 with few tasks) per SM.  Every CTA builds the list of
// chosen experts itself (at most 2048 assignments).  An expert's assignments
// are cut into groups of at most 8 (4 in very wide layers); a task is 16 weight
// rows (gate_up: 8 gate rows and the same 8 up rows, so the activation is local
// to a thread) of one group, over the whole length K; a CTA takes a contiguous
// run of tasks, so it reads contiguous rows and needs the activations of few
// groups.
//
// Weights.  A warp streams its tasks through its own ring of chunks (16 rows
// of 256 bytes of codes and their scales) in shared memory with cp.async, so
// no warp waits for another one's data; with few tasks 2, 4 or 8 warps split K
// and add their sums in a fixed order.  Rows are padded so that the fragment
// loads have no bank conflicts.
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
//
// Measured (512 experts, hidden 2048, inter 768, 10 experts a token): 64 tokens in
// NVFP4 235 us for the 952 MB of the experts chosen (4.0 TB/s), in MXFP8 294 us for
// 1.74 GB (5.9 TB/s); 16 in MXFP4 73 us; one in NVFP4 15.3 us.  What bounds it: of
// the 235 us the copies alone take 177 and the arithmetic alone 155 to 173, most of
// it conversions and scaling at two cycles an instruction; a token alone waits
// through the chain of dependent steps (list, first weights, rows, sums, twice).
#include "mxq_device.cuh"
#include "mxq_internal.h"
#include "mxq_mma.cuh"
#include "mxq.h"
#include <algorithm>

namespace mxq {

namespace {

// One chunk in shared memory: 16 rows of 256 bytes of codes, then the rows'
// scales.  With rows 272 bytes apart a fragment load (one word of each lane
// from 8 rows) touches every bank once; so do the scales, 48 bytes apart.
constexpr int kChunkBytes = 256;
constexpr int kPitch = kChunkBytes + 16;
constexpr int kScaleAt = 16 * kPitch;
constexpr int kScalePitch = 48;
constexpr int kSlotBytes = kScaleAt + 16 * kScalePitch;

struct MoeArgs {
    const uint16_t *x;          // gate_up: bf16 tokens [T, K]
    const float *hin;           // down: fp32 rows [A, K]
    const int32_t *ids;         // [A]
    const float *w;             // down: [A]
    const uint8_t *codes;       // [E, rows, K * bits / 8]
    const void *scales;
    const float *s2;            // NVFP4: [E]
    float *out;                 // gate_up: h [A, I]; down: z [A, H]
    uint16_t *y;                // down that sums itself: y [T, H]
    uint32_t *status;
    uint64_t expert_bytes;      // codes of one expert
    uint64_t expert_scales;     // scales of one expert (bytes)
    uint32_t row_bytes;         // codes of one row
    uint32_t row_scales;        // scales of one row (bytes); block-FP8: of one row of blocks
    uint32_t A, T, topk, E, K;
    uint32_t group;             // assignments of a group: 8, or 4 where 8 rows do not fit the stage
    uint32_t nrows;             // rows of an output: I or H
    uint32_t tiles;             // tasks of a group
    uint32_t chunks;            // chunks of a row
    uint32_t kslog;             // log2 of the warps that share a task
    uint32_t cap;               // activation rows the stage holds
    uint32_t xstride;           // bytes of a staged row
    uint32_t zs_at;             // where z lies behind the partial sums (floats)
    FastDiv tilesdiv, topkdiv, griddiv;
};

template <int FMT>
struct Fmt {
    static constexpr bool fp4 = FMT == MXQ_FMT_NVFP4 || FMT == MXQ_FMT_MXFP4;
    static constexpr int group_bytes = fp4 ? 64 : 128;                    // of 128 codes of a row
    static constexpr int chunk_k = 128 * kChunkBytes / group_bytes;       // values of a row in a chunk
    // scale bytes of 128 values of a row, and the bytes a lane copies at a time
    static constexpr int sbytes = FMT == MXQ_FMT_NVFP4 ? 8 : 4;
    static constexpr int schunk = sbytes * (kChunkBytes / group_bytes);   // of a chunk
};

// The chosen experts.  list: assignments sorted by expert; group g holds
// list[start[g] .. start[g + 1]) of expert expert[g], at most MoeArgs::group.
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
    uint32_t v = lead ? (((n + a.group - 1) / a.group) << 16) | n : 0u;
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
        if (rank % a.group == 0) {
            r.start[(base >> 16) + rank / a.group] = (uint16_t)((base & 0xFFFFu) + rank);
            r.expert[(base >> 16) + rank / a.group] = (uint16_t)id;
        }
    }
    if (lane == 0)
        r.start[total >> 16] = (uint16_t)(total & 0xFFFFu);
    return total >> 16;
}

// Up to 128: several lanes an assignment count the keys (expert, number) below its
// own, which is its place in the list, and those of lower experts; the places
// where groups begin are numbered by votes.  A layer of 84 assignments takes
// 9.9 us with it and 12.0 with route_block, one of 216 16.0 and 15.2.
template <int kWarps>
__device__ __forceinline__ uint32_t route_ranks(const MoeArgs &a, const Route &r, uint32_t *buf, uint32_t *wsum)
{
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    constexpr uint32_t none = 0xFFFFu, most = 128;
    static_assert(kWarps * 32 >= 4 * most, "four lanes an assignment");
    uint16_t *first = reinterpret_cast<uint16_t *>(buf + most);     // by place: the expert where a group begins
    const uint32_t lg = a.A <= 64u ? 3u : 2u, i = tid >> lg, part = tid & ((1u << lg) - 1u);
    bool valid = false;
    if (tid < most) {
        const int id = tid < a.A ? a.ids[tid] : -1;
        valid = id >= 0 && id < (int)a.E;
        if (id >= (int)a.E)
            atomicOr(a.status, MXQ_DEV_INVALID_EXPERT);
        buf[tid] = ((valid ? (uint32_t)id : none) << 16) | tid;
    }
    const uint32_t n = (uint32_t)__syncthreads_count(valid);
    const uint32_t key = buf[i & (most - 1u)], expert = key >> 16, low = expert << 16;
    uint32_t pos = 0, below = 0;
    for (uint32_t q = part; q < (a.A + 3u) / 4u; q += 1u << lg) {
        const uint4 k = *reinterpret_cast<const uint4 *>(buf + q * 4u);
        pos += (k.x < key) + (k.y < key) + (k.z < key) + (k.w < key);
        below += (k.x < low) + (k.y < low) + (k.z < low) + (k.w < low);
    }
    for (uint32_t o = 1; o < 1u << lg; o <<= 1) {
        pos += __shfl_xor_sync(0xFFFFFFFFu, pos, o);
        below += __shfl_xor_sync(0xFFFFFFFFu, below, o);
    }
    if (part == 0 && i < a.A && expert != none) {
        r.list[pos] = (uint16_t)i;
        first[pos] = (uint16_t)((pos - below) % a.group == 0 ? expert : none);
    }
    __syncthreads();
    const uint32_t e = tid < n ? first[tid] : none, vote = __ballot_sync(0xFFFFFFFFu, e != none);
    if (lane == 0)
        wsum[warp] = __popc(vote);
    __syncthreads();
    uint32_t at = __popc(vote & ((1u << lane) - 1u)), total = 0;
#pragma unroll
    for (uint32_t w = 0; w < most / 32; ++w) {
        at += w < warp ? wsum[w] : 0u;
        total += wsum[w];
    }
    if (e != none) {
        r.start[at] = (uint16_t)tid;
        r.expert[at] = (uint16_t)e;
    }
    if (tid == 0)
        r.start[total] = (uint16_t)n;
    __syncthreads();
    return total;
}

// More: ids, then counts and places of the experts in shared memory (E words
// at `cnt`), a scan, and a scatter.  The order of a group's assignments is
// free (each is a column of its own), but an expert's groups have to be the
// same in every CTA, so the list of an expert with more than one is put in
// ascending order.
template <int kWarps>
__device__ __forceinline__ uint32_t route_block(const MoeArgs &a, const Route &r, uint32_t *cnt, uint32_t *wsum)
{
    constexpr uint32_t kThreads = 32 * kWarps;
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    constexpr uint32_t none = 0xFFFFu;
    uint16_t *ids = reinterpret_cast<uint16_t *>(cnt + a.E);
    for (uint32_t i = tid; i < a.A; i += kThreads) {
        const int id = a.ids[i];
        if (id >= (int)a.E)
            atomicOr(a.status, MXQ_DEV_INVALID_EXPERT);
        ids[i] = (uint16_t)(id >= 0 && id < (int)a.E ? (uint32_t)id : none);
    }
    for (uint32_t e = tid; e < a.E; e += kThreads)
        cnt[e] = 0u;
    __syncthreads();
    for (uint32_t i = tid; i < a.A; i += kThreads)
        if (ids[i] != none)
            atomicAdd(&cnt[ids[i]], 1u);
    __syncthreads();
    // groups (high half) and assignments of the experts below
    const uint32_t per = (a.E + kThreads - 1) / kThreads, e0 = min(tid * per, a.E), e1 = min(e0 + per, a.E);
    uint32_t own = 0;
    for (uint32_t e = e0; e < e1; ++e)
        own += (((cnt[e] + a.group - 1) / a.group) << 16) | cnt[e];
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
#pragma unroll
    for (uint32_t i = 0; i < kWarps; ++i) {
        if (i < warp)
            v += wsum[i];
        total += wsum[i];
    }
    v -= own;
    bool more = false;
    for (uint32_t e = e0; e < e1; ++e) {
        const uint32_t n = cnt[e];
        cnt[e] = (n << 16) | (v & 0xFFFFu);
        more |= n > a.group;
        for (uint32_t i = 0; i < n; i += a.group) {
            r.start[v >> 16] = (uint16_t)(v & 0xFFFFu);
            r.expert[v >> 16] = (uint16_t)e;
            v += (1u << 16) + min(n - i, a.group);
        }
    }
    if (tid == 0)
        r.start[total >> 16] = (uint16_t)(total & 0xFFFFu);
    more = __syncthreads_or(more);
    for (uint32_t i = tid; i < a.A; i += kThreads)
        if (ids[i] != none)
            r.list[atomicAdd(&cnt[ids[i]], 1u) & 0xFFFFu] = (uint16_t)i;
    __syncthreads();
    if (more) {
        constexpr int most = (int)((kMoeMaxAssignments + kThreads - 1) / kThreads);
        uint32_t val[most], to[most];
#pragma unroll
        for (int k = 0; k < most; ++k) {
            const uint32_t pos = tid + k * kThreads;
            to[k] = none;
            if (pos < (total & 0xFFFFu)) {
                val[k] = r.list[pos];
                const uint32_t c = cnt[ids[val[k]]], n = c >> 16, end = c & 0xFFFFu;    // past its last place now
                if (n > a.group) {
                    to[k] = end - n;
                    for (uint32_t j = end - n; j < end; ++j)
                        to[k] += r.list[j] < val[k];
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < most; ++k)
            if (to[k] != none)
                r.list[to[k]] = (uint16_t)val[k];
        __syncthreads();
    }
    return total >> 16;
}

// Where four values lie in a staged row.  4-bit formats: in order; a lane's
// word holds 8 codes.  8-bit formats: a lane has one word (4 codes) of two
// neighbouring pieces, so of every 32 values the quads 0, 4, 1, 5, ... follow
// one another.
template <int FMT>
__device__ __forceinline__ uint32_t staged(uint32_t k)
{
    const uint32_t q = (k >> 2) & 7u;
    return Fmt<FMT>::fp4 ? k * 2u : ((k & ~31u) + ((q & 3u) * 2u + (q >> 2)) * 4u) * 2u;
}

// One warp: row `a` of the activations -> f16 at `dst`, its inverse factor
// returned.
template <int FMT, bool GATE_UP>
__device__ __forceinline__ float stage_row(const MoeArgs &g, uint32_t a, char *dst, uint32_t lane)
{
    uint32_t m = 0;
    if (GATE_UP) {
        const uint16_t *src = g.x + (uint64_t)fastdiv(a, g.topkdiv) * g.K;
#pragma unroll 8
        for (uint32_t k = lane * 8u; k < g.K; k += 256u) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src + k));
            uint32_t q = absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(0u, v.x), v.y), v.z), v.w);
            m = max(m, fold_halves(q));
        }
        m = __reduce_max_sync(0xFFFFFFFFu, m) << 16;
        if (m >= 0x7F800000u && lane == 0)
            atomicOr(g.status, MXQ_DEV_NONFINITE_INPUT);
        const float f = row_factor(m);
#pragma unroll 8
        for (uint32_t k = lane * 8u; k < g.K; k += 256u) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src + k));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                h[i] = half2_bits(bf16_lo(w[i]) * f, bf16_hi(w[i]) * f);
            if (Fmt<FMT>::fp4)
                *reinterpret_cast<uint4 *>(dst + k * 2u) = make_uint4(h[0], h[1], h[2], h[3]);
            else {
                *reinterpret_cast<uint2 *>(dst + staged<FMT>(k)) = make_uint2(h[0], h[1]);
                *reinterpret_cast<uint2 *>(dst + staged<FMT>(k + 4u)) = make_uint2(h[2], h[3]);
            }
        }
        return 1.0f / f;
    }
    const float *src = g.hin + (uint64_t)a * g.K;
#pragma unroll 6
    for (uint32_t k = lane * 4u; k < g.K; k += 128u) {
        const float4 v = *reinterpret_cast<const float4 *>(src + k);
        m = max(max(m, max(__float_as_uint(fabsf(v.x)), __float_as_uint(fabsf(v.y)))),
                max(__float_as_uint(fabsf(v.z)), __float_as_uint(fabsf(v.w))));
    }
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    const float f = row_factor(m >= 0x7F800000u ? 0u : m);
#pragma unroll 6
    for (uint32_t k = lane * 4u; k < g.K; k += 128u) {
        const float4 v = *reinterpret_cast<const float4 *>(src + k);
        *reinterpret_cast<uint2 *>(dst + staged<FMT>(k)) =
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

template <int FMT, bool GATE_UP, int D, int kWarps, bool SPLIT, bool WHOLE>
__global__ void __launch_bounds__(32 * kWarps, 16 / kWarps)
moe_kernel(const MoeArgs a)
{
    constexpr uint32_t kThreads = 32 * kWarps;
    using F = Fmt<FMT>;
    extern __shared__ __align__(128) char smem[];
    __shared__ uint32_t wsum[kWarps];
    __shared__ uint32_t groups_s;
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5, g8 = lane >> 2, t4 = lane & 3u;
    if (GATE_UP)
        cudaGridDependencySynchronize();     // whatever ran before may have written what this reads
    // shared memory: rings, activation rows, row factors, lists, partial sums
    char *ring = smem + warp * (D * kSlotBytes);
    char *xs = smem + kWarps * D * kSlotBytes;
    float *xf = reinterpret_cast<float *>(xs + (a.cap + 1u) * a.xstride);
    float *part = xf + ((a.cap + 3u) & ~3u);
    Route r;
    r.list = reinterpret_cast<uint16_t *>(part + kWarps * 128);
    r.start = r.list + a.A;
    r.expert = r.start + a.A + 1;
    // WHOLE: z of the CTA's tiles, [tile][assignment][16 rows]
    float *zs = part + kWarps * 128 + a.zs_at;
    if (kWarps < 16 || a.A <= 32u) {
        if (warp == 0) {
            const uint32_t n = route_warp(a, r, lane);
            if (lane == 0)
                groups_s = n;
        }
        __syncthreads();
        r.groups = groups_s;
    } else if (a.A <= 128u)
        r.groups = route_ranks<16>(a, r, reinterpret_cast<uint32_t *>(xs), wsum);
    else
        r.groups = route_block<kWarps>(a, r, reinterpret_cast<uint32_t *>(xs), wsum);
    for (uint32_t k = tid * 16u; k < a.xstride; k += kThreads * 16u)
        *reinterpret_cast<uint4 *>(xs + a.cap * a.xstride + k) = make_uint4(0u, 0u, 0u, 0u);
    // this CTA's run of tasks
    const uint32_t ntask = WHOLE ? a.tiles : r.groups * a.tiles;
    uint32_t t0 = fastdiv(ntask * blockIdx.x, a.griddiv), t1 = fastdiv(ntask * (blockIdx.x + 1), a.griddiv);
    const uint32_t tile0 = t0, ntile = t1 - t0;      // WHOLE: of tiles, each with all groups
    if (WHOLE) {
        t0 = 0;
        t1 = ntile * r.groups;
    }
    auto split = [&](uint32_t task, uint32_t &grp, uint32_t &tile) {
        if (WHOLE) {
            tile = task / r.groups;
            grp = task - tile * r.groups;
            tile += tile0;
        } else {
            grp = fastdiv(task, a.tilesdiv);
            tile = task - grp * a.tiles;
        }
    };
    const uint32_t lg = SPLIT ? a.kslog : 0u, ks = 1u << lg, teams = kWarps >> lg, team = warp >> lg, q = warp & (ks - 1u);
    const uint32_t c0 = (a.chunks * q) >> lg, c1 = (a.chunks * (q + 1)) >> lg;

    const uint32_t half = GATE_UP ? a.nrows : 8u;    // distance of the second 8 rows from the first
    const uint32_t tile_rows = GATE_UP ? 8u : 16u;
    const uint32_t piece = lane & 7u, half8 = (t4 >> 1) * 8u;
    const uint32_t ring_s = smem_addr(ring);
    // scale pieces of a row: 4 (4-bit formats: the lanes cover 8 rows, twice) or 2
    constexpr uint32_t spieces = F::fp4 ? 4 : 2;
    const uint32_t srow = lane / spieces, spiece = lane % spieces;
    Walk p;
    p.task = t0 + team;
    p.ch = c0;
    auto locate = [&]() {
        uint32_t grp, tile;
        split(p.task, grp, tile);
        const uint32_t e = r.expert[grp];
        const uint32_t r0 = tile * tile_rows;
        p.code = a.codes + e * a.expert_bytes + (uint64_t)(r0 + (lane >> 3)) * a.row_bytes + piece * 16u;
        const char *se = static_cast<const char *>(a.scales) + e * a.expert_scales;
        if (FMT == MXQ_FMT_FP8_BLOCK)      // lanes 0-1 and 2-3: the block rows of the two halves
            p.scale = se + (uint64_t)((r0 + ((lane >> 1) & 1u) * half) >> 7) * a.row_scales;
        else                               // pieces of sbytes, spieces to a row
            p.scale = se + (uint64_t)(r0 + (srow & 7u) + (srow >> 3) * half) * a.row_scales;
    };
    const uint32_t code_dst = ring_s + (lane >> 3) * kPitch + piece * 16u;
    const uint32_t scale_dst = ring_s + kScaleAt + (FMT == MXQ_FMT_FP8_BLOCK ? (lane >> 1) * 8u : srow) * kScalePitch +
                               spiece * F::sbytes;
    const uint64_t r4 = 4ull * a.row_bytes, hb = (uint64_t)half * a.row_bytes;
    const uint64_t s8 = (uint64_t)half * a.row_scales;
    auto issue = [&](uint32_t slot) {
        if (p.task < t1) {
            const uint32_t dst = code_dst + slot * kSlotBytes, sd = scale_dst + slot * kSlotBytes;
            const uint32_t left = a.row_bytes - p.ch * kChunkBytes;      // of the row, from this chunk on
            const uint8_t *q0 = p.code + p.ch * kChunkBytes, *q1 = q0 + r4, *q2 = q0 + hb, *q3 = q2 + r4;
            if (piece * 16u < left) {
                cp16(dst, q0);
                cp16(dst + 4 * kPitch, q1);
                cp16(dst + 8 * kPitch, q2);
                cp16(dst + 12 * kPitch, q3);
            }
            if (piece * 16u + 128u < left) {
                cp16(dst + 128, q0 + 128);
                cp16(dst + 4 * kPitch + 128, q1 + 128);
                cp16(dst + 8 * kPitch + 128, q2 + 128);
                cp16(dst + 12 * kPitch + 128, q3 + 128);
            }
            const char *s = p.scale + p.ch * F::schunk + spiece * F::sbytes;
            if (spiece * F::group_bytes < left) {
                if (F::fp4) {                       // rows 0-7, rows 8-15
                    cp_small<F::sbytes>(sd, s);
                    cp_small<F::sbytes>(sd + 8 * kScalePitch, s + s8);
                } else if (FMT == MXQ_FMT_MXFP8 || lane < 4u)
                    cp_small<4>(sd, s);
            }
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
    if (D == 2)
        issue(0);
    if (!GATE_UP)
        cudaGridDependencySynchronize();     // h is written by the launch before
    cudaTriggerProgrammaticLaunchCompletion();

    uint32_t slot = 0, pos = t0, task = t0 + team;
    while (pos < t1) {
        // activations of as many groups as the stage holds
        const uint32_t g0 = WHOLE ? 0u : fastdiv(pos, a.tilesdiv), row0 = r.start[g0];
        uint32_t gl = WHOLE ? r.groups : g0 + 1;
        const uint32_t gend = WHOLE ? gl : fastdiv(t1 - 1u, a.tilesdiv) + 1u;
        while (gl < gend && (uint32_t)r.start[gl + 1] - row0 <= a.cap)
            ++gl;
        const uint32_t end = WHOLE ? t1 : min(t1, gl * a.tiles), nr = (uint32_t)r.start[gl] - row0;
        __syncthreads();
        for (uint32_t i = warp; i < nr; i += kWarps) {
            const float f = stage_row<FMT, GATE_UP>(a, r.list[row0 + i], xs + i * a.xstride, lane);
            if (lane == 0)
                xf[i] = f;
        }
        __syncthreads();
        for (; task < end; task += teams) {
            uint32_t grp, tile;
            split(task, grp, tile);
            const uint32_t first = r.start[grp], cnt = r.start[grp + 1] - first;
            // columns without an assignment read the row of zeros
            const char *xrow = xs + (g8 < cnt ? first - row0 + g8 : a.cap) * a.xstride + t4 * 16u;
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f}, acc2[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            for (uint32_t ch = c0; ch < c1; ++ch) {
                if (D == 1) {
                    __syncwarp();
                    issue(0);
                    cp_wait<0>();
                    __syncwarp();
                } else {
                    cp_wait<0>();
                    __syncwarp();
                    issue(slot ^ 1u);            // the slot read in the step before
                }
                // this lane's words of rows g8 and g8 + 8, and their scales
                const char *cw = ring + slot * kSlotBytes + g8 * kPitch + t4 * 4u;
                const char *sb = ring + slot * kSlotBytes + kScaleAt +
                                 (FMT == MXQ_FMT_FP8_BLOCK ? 0u : g8 * kScalePitch);
                slot = D == 2 ? slot ^ 1u : 0u;
                const char *xk = xrow + ch * (F::chunk_k * 2u);
                const uint32_t groups = min((uint32_t)F::chunk_k, a.K - ch * F::chunk_k) >> 7;
#pragma unroll 2
                for (uint32_t hk = 0; hk < groups; ++hk, cw += F::group_bytes, sb += F::sbytes, xk += 256) {
                    float d0[4], d1[4], c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    uint32_t s0[4], s1[4];
                    if (FMT == MXQ_FMT_NVFP4) {
                        // pairs of scales of 32 values, the one of this lane's 16 first
                        const uint2 n0 = lds64(sb), n1 = lds64(sb + 8 * kScalePitch);
                        e4m3x4_unpack(n0.x >> half8, s0[0], s0[1]);
                        e4m3x4_unpack(n0.y >> half8, s0[2], s0[3]);
                        e4m3x4_unpack(n1.x >> half8, s1[0], s1[1]);
                        e4m3x4_unpack(n1.y >> half8, s1[2], s1[3]);
                    } else if (FMT == MXQ_FMT_FP8_BLOCK) {
                        d0[0] = __uint_as_float(lds32(sb));
                        d1[0] = __uint_as_float(lds32(sb + 8 * kScalePitch));
                    } else {
                        ue8m0x4(lds32(sb), d0);
                        ue8m0x4(lds32(sb + 8 * kScalePitch), d1);
                    }
#pragma unroll
                    for (uint32_t u = 0; u < 4; ++u) {           // 32 values of a row
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
                        const uint4 b = lds128(xk + u * 64u);
                        if (FMT == MXQ_FMT_NVFP4) {
                            const uint32_t e0 = low2(s0[u]), e1 = low2(s1[u]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                p0[i] = hmul2_bits(p0[i], e0);
                                p1[i] = hmul2_bits(p1[i], e1);
                            }
                            mma16816(acc, p0[0], p1[0], p0[1], p1[1], b.x, b.y);
                            mma16816(acc2, p0[2], p1[2], p0[3], p1[3], b.z, b.w);
                            continue;
                        }
                        mma16816(c, p0[0], p1[0], p0[1], p1[1], b.x, b.y);
                        mma16816(c, p0[2], p1[2], p0[3], p1[3], b.z, b.w);
                        if (FMT == MXQ_FMT_FP8_BLOCK ? u == 3 : true) {      // a scale block is complete
                            const float f0 = d0[FMT == MXQ_FMT_FP8_BLOCK ? 0 : u];
                            const float f1 = d1[FMT == MXQ_FMT_FP8_BLOCK ? 0 : u];
                            acc[0] = fmaf(c[0], f0, acc[0]);
                            acc[1] = fmaf(c[1], f0, acc[1]);
                            acc[2] = fmaf(c[2], f1, acc[2]);
                            acc[3] = fmaf(c[3], f1, acc[3]);
                            c[0] = c[1] = c[2] = c[3] = 0.0f;
                        }
                    }
                }
            }
            if (FMT == MXQ_FMT_NVFP4)   // two chains of products
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[i] += acc2[i];
            if (SPLIT && ks > 1) {       // the team's partial sums, in warp order
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
                            float *o = WHOLE ? zs + ((tile - tile0) * a.A + as) * 16u + g8
                                             : a.out + (uint64_t)as * a.nrows + tile * 16u + g8;
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
    if (WHOLE) {        // y[t] = sum over the token's experts of z, in their order; 2 columns a thread
        __syncthreads();
        for (uint32_t i = tid; i < ntile * a.T * 8u; i += kThreads) {
            const uint32_t row = i >> 3, tl = row / a.T, t = row - tl * a.T, c = (i & 7u) * 2u;
            float2 s = make_float2(0.0f, 0.0f);
            for (uint32_t j = 0; j < a.topk; ++j) {
                const int id = a.ids[t * a.topk + j];
                if (id < 0 || id >= (int)a.E)
                    continue;
                const float2 v = *reinterpret_cast<const float2 *>(zs + (tl * a.A + t * a.topk + j) * 16u + c);
                s.x += v.x;
                s.y += v.y;
            }
            *reinterpret_cast<__nv_bfloat162 *>(a.y + (uint64_t)t * a.nrows + (tile0 + tl) * 16u + c) =
                __floats2bfloat162_rn(s.x, s.y);
        }
    }
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

constexpr size_t kSmemHalf = 113 * 1024 - 256;
constexpr size_t kSmemMax = 227 * 1024 - 256;     // less the static words of the kernel

template <int FMT, bool GATE_UP, int D, int W, bool SPLIT, bool WHOLE = false>
cudaError_t run(const MoeArgs &a, size_t smem, int ctas, cudaStream_t s)
{
    const auto k = moe_kernel<FMT, GATE_UP, D, W, SPLIT, WHOLE>;
    // The limit belongs to the kernel, not to the launch: always the largest, so that
    // calls of other sizes from other threads set the same.
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)(W == 8 ? kSmemHalf : kSmemMax));
    if (e != cudaSuccess)
        return e;
    return launch_dependent(k, dim3((unsigned)ctas), 32 * W, smem, s, a);
}

// `summed` is set where the down launch has written y itself.
template <int FMT, bool GATE_UP>
cudaError_t moe_gemm(MoeArgs a, int ctas, cudaStream_t s, bool &summed)
{
    a.row_bytes = Fmt<FMT>::fp4 ? a.K / 2 : a.K;
    a.row_scales = FMT == MXQ_FMT_NVFP4 ? a.K / 16 : FMT == MXQ_FMT_FP8_BLOCK ? a.K / 128 * 4 : a.K / 32;
    const uint64_t rows = GATE_UP ? 2ull * a.nrows : a.nrows;
    a.expert_bytes = rows * a.row_bytes;
    a.expert_scales = (FMT == MXQ_FMT_FP8_BLOCK ? rows / 128 : rows) * a.row_scales;
    a.tiles = a.nrows / (GATE_UP ? 8 : 16);
    a.tilesdiv = make_fastdiv(a.tiles);
    a.topkdiv = make_fastdiv(a.topk);
    a.griddiv = make_fastdiv((uint32_t)ctas);
    a.chunks = (a.K + Fmt<FMT>::chunk_k - 1) / Fmt<FMT>::chunk_k;
    a.xstride = a.K * 2 + 64;       // 64 mod 128: the rows of a fragment load fall on different banks
    const uint64_t most_tasks = (uint64_t)a.A * a.tiles;    // were all assignments of different experts
    // Shared memory of a CTA of `warps` whose rings are `depth` chunks and whose
    // stage has `rows` activation rows, one of zeros and room to round them up.
    const auto need = [&](size_t warps, size_t depth, size_t rows) {
        return warps * (depth * kSlotBytes + 128 * 4) + (3 * (size_t)a.A + 2) * 2 + 64 +
               (rows + 1) * ((size_t)a.xstride + 4) + 16;
    };
    // The stage takes what `all` bytes leave, up to 64 rows (with 16 warps at
    // least 20 KB in all: ids and expert counts lie there first); an expert's
    // assignments are taken 8 at a time, or 4 where 8 rows do not fit.  Warps
    // that share a task: doubled while every warp of the grid still gets at most
    // one and each has a chunk.  Not by the experts really chosen: a token's sums
    // are then added in the same order whatever its company chose.
    const auto plan = [&](size_t warps, size_t depth, size_t all) {
        a.cap = (uint32_t)std::min<size_t>((all - need(warps, depth, 0)) / (a.xstride + 4), 64);
        a.group = a.cap >= 8 ? 8 : 4;
        a.kslog = 0;
        while (a.kslog < 3 && (2u << a.kslog) <= a.chunks && (most_tasks * 2 << a.kslog) <= (uint64_t)ctas * warps)
            ++a.kslog;
        return need(warps, depth, a.cap);
    };
    // At most a task a warp: CTAs of 8 warps and half the shared memory, so that the
    // next launch fetches its first weights meanwhile (5 tokens of a tiny layer
    // 7.9 us, with 16 warps 9.6; up to two tasks a warp a token of 10 experts takes
    // 15.8 us, so 15.4).
    const bool few = a.A <= 32 && most_tasks <= (uint64_t)ctas * 8;
    // And, where a CTA's tiles of the down product make about a task a warp (as
    // many groups as assignments or experts) and the rows are short, it takes them
    // for all groups and adds up y itself: two launches instead of three, which
    // saves 2.5 us of the caller's time (14.9 -> 12.3 for 5 tokens of a tiny layer,
    // 7.5 on the GPU either way; one token of 2 experts 7.5 -> 6.7 on the GPU).
    // With more tasks the other way is faster: 16.0 against 18.7 us for a token of
    // 10 experts, and 14.3 against 15.3 with rows of 8 chunks.
    const size_t per = (a.tiles + ctas - 1) / ctas, zs = per * a.A * 16 * 4;
    const size_t tasks = per * std::min(a.A, a.E);
    if (!GATE_UP && few && tasks <= 8 && a.chunks <= 5 && need(8, 2, a.A) + 16 + zs <= kSmemHalf) {
        plan(8, 2, kSmemHalf);                      // the warps that share a task as in the other way
        a.cap = a.A;
        a.group = 8;
        a.zs_at = (3 * a.A + 2 + 7) / 8 * 4;        // behind the lists
        summed = true;
        return run<FMT, GATE_UP, 2, 8, true, !GATE_UP>(a, need(8, 2, a.A) + 16 + zs, ctas, s);
    }
    if (few && need(8, 2, 4) <= kSmemHalf)
        return run<FMT, GATE_UP, 2, 8, true>(a, plan(8, 2, kSmemHalf), ctas, s);
    // Rings of 2 chunks a warp; in layers too wide for that and 4 rows, of 1.
    // Tasks of one warp each are a kernel of their own: without the limits of a
    // share 16 MXFP4 tokens take 72.5 us, with them 77.8.
    if (need(16, 2, 4) > kSmemMax)
        return run<FMT, GATE_UP, 1, 16, true>(a, plan(16, 1, kSmemMax), ctas, s);
    const size_t smem = plan(16, 2, kSmemMax);
    return a.kslog ? run<FMT, GATE_UP, 2, 16, true>(a, smem, ctas, s) : run<FMT, GATE_UP, 2, 16, false>(a, smem, ctas, s);
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
    a.T = (uint32_t)m.T;
    a.y = m.y;
    a.topk = (uint32_t)m.topk;
    a.E = (uint32_t)m.experts;
    a.codes = m.gu_codes;
    a.scales = m.gu_scales;
    a.s2 = m.gu_s2;
    a.out = m.h;
    a.K = (uint32_t)m.hidden;
    a.nrows = (uint32_t)m.inter;
    bool summed = false;
    cudaError_t e = moe_gemm<FMT, true>(a, sms, s, summed);
    if (e != cudaSuccess)
        return e;
    a.codes = m.dn_codes;
    a.scales = m.dn_scales;
    a.s2 = m.dn_s2;
    a.out = m.z;
    a.K = (uint32_t)m.inter;
    a.nrows = (uint32_t)m.hidden;
    e = moe_gemm<FMT, false>(a, sms, s, summed);
    if (e != cudaSuccess || summed)
        return e;
    return launch_dependent(moe_combine_kernel, dim3((unsigned)((m.hidden + 511) / 512), (unsigned)m.T), 128, 0, s,
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
