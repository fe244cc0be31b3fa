// attention_rows.cu -- attention over a quantized cache where a sequence has few
// rows: decoding, guessed tokens (sm_100a).  The read of the cache is the work.
//
// A tile is up to 8 rows (where no sequence of the call has more) or 16 of one sequence
// and key/value head, a step 32 keys; attention.cuh divides them.  A CTA has 4 warps,
// which take turns of the steps of a tile, each with its own running maximum, sum and
// output, joined at the end (in the order of the warps).  Where there are few tiles and a
// warp has few turns, a cluster of CTAs takes each tile instead (CLUSTER), a run of its
// steps a CTA, and the parts are joined through the CTAs' shared memory: nothing is
// divided and no second launch is needed, which is most of a short call's time.
//
// Codes go from global memory to a warp's own two stages of shared memory by
// cp.async and from there, decoded, into the left operands of mma.sync m16n8k16 (f16,
// fp32 sums): 16 keys of S^T = K Q^T, 16 columns of O^T = V^T P^T, so that 8 rows waste
// nothing.  The order of a head's dimension inside a product is free, so a lane takes a
// contiguous run of every key's codes, and a contiguous run of the values' columns;
// pairs of keys are put together a byte (or nibble) at a time before they are decoded, so
// the values need no transposition; the weights are turned by movmatrix.
//
// Bound: the arithmetic of the decoding beside HBM.  64 sequences of up to 32768 tokens,
// 2 key/value heads of 128 for 16 query heads, one token each: MXFP8 67 us (328 MB, 4.9
// TB/s, 75 % of the measured copy rate), NVFP4 63 us, heads of 64 57 us, 32 sequences with
// heads of 256 73 us; with keys as right operands and rows as 16 left ones MXFP8 took 98 us.
// 12 of up to 16384, heads of 256, 4 tokens each (two tiles of 16 rows), NVFP4: 41 us.  One
// sequence of 5000: 11 us, 17 us without clusters; beyond 8 turns a warp the division
// wins (12 of 16384 as above by clusters 120 us, divided 59 then).  Two warps to a turn, each
// with half of its keys' scores and half of the columns, so that 32 rows fit: 59 us for
// the 12 of 16384 against 46, the barrier of a turn costs more than a second decoding.
//
// Precision.  E2M1 times its E4M3 scale is exact in f16.  E4M3 codes (MXFP8) are
// multiplied in f16 by their block's power of two relative to the largest of the
// warp's 32 keys, 2^7 at most: exact while the blocks' maxima lie within 2^22 of one
// another, below that off by 2^-25 / 57344 of the largest, and zero from 2^-32 on.  The
// largest one's power itself multiplies the scores in fp32.  Values: relative to a
// reference of the warp and the 32 columns of the block (ValueRef), so columns do not
// share it; it may stand one above the 32 keys' largest, exact within 2^21 then.  Queries are held in f16 times a power of two of the row (as the
// layer's tokens, moe.cu); weights are rounded to f16's 11 bits, an eighth of the bf16
// result's own step; scores, references, sums and outputs are fp32.
#include "attention.cuh"
#include "mxq_cluster.cuh"
#include "mxq_mma.cuh"
#include <algorithm>

namespace mxq {

namespace {

constexpr uint32_t kKeys = 32, kLog = 5;    // keys of a step
constexpr uint32_t kWarps = 4;
constexpr uint32_t kMostSteps = 4096;       // of a piece: 2^15 keys a warp
constexpr uint32_t kClusterTurns = 8;       // most turns of a warp, of a tile that a cluster takes

template <int FMT, int D, int NT>
struct Shape {
    static constexpr uint32_t R = 8 * NT;                       // rows of a tile
    static constexpr bool fp4 = FMT == MXQ_FMT_NVFP4;
    static constexpr uint32_t row = fp4 ? D / 2 : D;            // bytes of a key's codes
    static constexpr uint32_t blocks = fp4 ? D / 16 : D / 32;   // and of its scales
    static constexpr uint32_t codes = kKeys * row, scales = kKeys * blocks;
    static constexpr uint32_t stage = 2 * (codes + scales);     // k codes, v codes, k scales, v scales
    static constexpr uint32_t ring = 2 * stage;                 // of a warp
    static constexpr bool q_regs = D * NT <= 128;                    // queries in registers
    // Bytes of a lane's run of a query row in shared memory, and of a row: 8 lanes' loads of
    // 16 bytes (four runs of two rows) touch every bank once.
    static constexpr uint32_t q_run = D / 2 + (D == 64 ? 0 : 32), q_pitch = 4 * q_run + 16;
    static constexpr uint32_t outs = R * (D + 4) * 4;       // a warp's outputs, when they are joined
    static constexpr uint32_t smem = kWarps * ring + R * q_pitch;
    static constexpr uint32_t all = smem > kWarps * outs ? smem : kWarps * outs;
    static constexpr uint32_t most = (D == 64 ? 4 : D == 128 ? 3 : 2) + (NT == 1 ? 1 : 0);      // CTAs of an SM, by registers
    static constexpr uint32_t room = (227 * 1024) / (all + 2048);           // and by shared memory
    static constexpr uint32_t fit = room < most ? room : most;
    static_assert(fit <= 5 && fit * R <= 64, "the workspace");
};

// Byte `off` of a stage's codes in shared memory: 16-byte pieces are permuted in
// their 128-byte line so that the reads of 8 lanes (keys: pieces of neighbouring rows;
// values: the same piece of every other row) touch every bank once.
template <uint32_t ROW>
__device__ __forceinline__ uint32_t swizzle(uint32_t off)
{
    const uint32_t line = off >> 7;
    uint32_t m;
    if (ROW == 256)
        m = ((line >> 1) & 7u) ^ ((line & 1u) << 1);
    else if (ROW == 128)
        m = line & 7u;
    else if (ROW == 64)
        m = (line & 3u) << 1;
    else
        m = (line & 1u) << 1;
    return off ^ (m << 4);
}

// 8 x 8 halves: lane 4 r + c has (r, 2 c) and (r, 2 c + 1), and gets (2 c, r) and (2 c + 1, r).
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// What the pieces of a tile before this one left in `part` is added to the warps' outputs
// `outs` and to their references and sums `stat` (the first warp's are then all).  All threads,
// between barriers.
template <uint32_t R, int D, uint32_t OUTS>
__device__ __noinline__ void add_earlier(float *outs, float *stat, const float *part)
{
    constexpr uint32_t kThreads = 32 * kWarps;
    static_assert(R <= kThreads, "a row a thread");
    const uint32_t tid = threadIdx.x;
    for (uint32_t i = tid; i < R * (D + 4) / 4; i += kThreads) {      // the row's reference and sum as columns D and on
        const uint32_t r = i / (D / 4 + 1), d = i % (D / 4 + 1) * 4;
        const float2 st = *reinterpret_cast<const float2 *>(part + R * D + r * 2);
        float m = st.x, own = 0.0f;
#pragma unroll
        for (uint32_t w = 0; w < kWarps; ++w)
            m = fmaxf(m, stat[w * R + r]);
#pragma unroll
        for (uint32_t w = 0; w < kWarps; ++w)
            own = fmaf(stat[(kWarps + w) * R + r], ex2(stat[w * R + r] - m), own);
        const float share = st.y * ex2(st.x - m), f = inverse(share + own), g = share * f, h = own * f;
        if (d == D) {
            outs[r * (D + 4) + D] = m;
            outs[r * (D + 4) + D + 1] = share + own;
            continue;
        }
        float4 v = *reinterpret_cast<const float4 *>(part + r * D + d);
        v = make_float4(v.x * g, v.y * g, v.z * g, v.w * g);
#pragma unroll
        for (uint32_t w = 0; w < kWarps; ++w) {
            float4 *at = reinterpret_cast<float4 *>(outs + w * OUTS + r * (D + 4) + d);
            const float4 x = *at;
            v = make_float4(fmaf(x.x, h, v.x), fmaf(x.y, h, v.y), fmaf(x.z, h, v.z), fmaf(x.w, h, v.w));
            *at = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        *reinterpret_cast<float4 *>(outs + r * (D + 4) + d) = v;
    }
    __syncthreads();
    if (tid < R) {
        const float top = outs[tid * (D + 4) + D], l = outs[tid * (D + 4) + D + 1];
#pragma unroll
        for (uint32_t w = 0; w < kWarps; ++w) {
            stat[w * R + tid] = w ? kLowest : top;
            stat[(kWarps + w) * R + tid] = w ? 0.0f : l;
        }
    }
    __syncthreads();
}

} // namespace

template <int FMT, int D, int NT, bool CLUSTER>
__global__ void __launch_bounds__(32 * kWarps, Shape<FMT, D, NT>::fit)
attention_rows_kernel(const __grid_constant__ AttArgs a)
{
    using S = Shape<FMT, D, NT>;
    constexpr uint32_t kRows = S::R;
    using W = Walk<kRows, kLog, kMostSteps>;
    constexpr uint32_t kThreads = 32 * kWarps;
    extern __shared__ __align__(128) char smem[];
    __shared__ Range range;
    __shared__ AttArgs sa;      // for functions out of line
    __shared__ W walks[kWarps];
    __shared__ __align__(16) float stat[2][kWarps][kRows];        // the warps' maxima and sums
    __shared__ __align__(16) float joint[2][kRows];               // the CTA's
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5, g8 = lane >> 2, t4 = lane & 3u;
    if (!CLUSTER && tid == 0)
        sa = a;
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();
    W &walk = walks[warp];
    uint32_t rank = 0, ranks = 1;
    bool more;
    if (CLUSTER) {
        asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
        asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
        const uint32_t c = blockIdx.x / ranks, tile = c % a.tiles, ch = c / a.tiles;
        W w;
        w.b = ch / a.c.heads;
        w.head = ch - w.b * a.c.heads;
        w.rt = tile;
        w.s = sequence(a, w.b);
        if (tile >= W::Div::tiles(w.s))
            return;             // all of the cluster
        w.steps = W::Div::steps(a, w.s, tile);
        w.keys = W::Div::keys(a, w.s, tile);
        w.k0 = a.extra + (uint32_t)((uint64_t)(w.steps - a.extra) * rank / ranks);
        w.k1 = a.extra + (uint32_t)((uint64_t)(w.steps - a.extra) * (rank + 1u) / ranks);
        w.begun = w.k0;
        w.left = 0;
        __syncwarp();
        if (lane == 0)
            walk = w;
        __syncwarp();
        more = true;
    } else {
        __syncthreads();
        find_range<W::Div>(sa, range);
        if (tid == 0)
            a.left[blockIdx.x].parts = 0u;
        more = W::begin(walk, sa, range);
    }

    const uint64_t once = once_policy();
    char *ring = smem + warp * S::ring;
    const uint32_t ring_s = smem_addr(ring);
    char *qs = smem + kWarps * S::ring;
    for (; more; more = !CLUSTER && W::next(walk, sa)) {
        const uint32_t first = walk.s.first, rows = walk.s.rows, tile = walk.rt, head = walk.head, b = walk.b;
        const int64_t pos0 = walk.s.len - walk.s.n;           // position of the sequence's first new token
        const uint32_t k0 = walk.from(a) << kLog, k1 = min(walk.to(a) << kLog, walk.keys);
        __syncthreads();
        // Pages of a turn's keys, as the table has them: 32 keys lie on one page, or on two of 16
        // tokens.  Looked up a turn before the copies are made, which are a turn ahead themselves.
        const bool short_pages = a.c.page_log == 4u;
        auto look = [&](uint32_t key, uint32_t (&page)[2]) {
            page[0] = key < k1 ? table_entry(a.c, b, key) : 0u;
            page[1] = short_pages && key + 16u < k1 ? table_entry(a.c, b, key + 16u) : page[0];
        };
        // One turn's copies: two runs of 16 keys, each contiguous.
        auto issue = [&](uint32_t key, uint32_t slot, const uint32_t (&page)[2]) {
            if (key < k1) {
                if (page[0] >= a.c.pages || page[1] >= a.c.pages)
                    atomicOr(a.c.status, MXQ_DEV_INVALID_PAGE);
                const uint32_t mask = (1u << a.c.page_log) - 1u, st = ring_s + slot * S::stage;
                const uint32_t keys0 = page[0] < a.c.pages ? k1 - key : 0u, keys1 = page[1] < a.c.pages ? k1 - key : 0u;
                uint64_t at[2];         // rows of codes of keys 0 and 16 (0 where they are not read)
                at[0] = keys0 ? (((uint64_t)page[0] * a.c.heads + head) << a.c.page_log) + (key & mask) : 0ull;
                at[1] = keys1 > 16u ? (((uint64_t)page[1] * a.c.heads + head) << a.c.page_log) + ((key + 16u) & mask) : 0ull;
                constexpr uint32_t pieces = S::row / 16;        // of a key's codes
                static_assert(pieces * 16 % 32 == 0 && S::scales % 32 == 0, "a copy of the warp stays in a run");
                if (keys0 >= kKeys && keys1 >= kKeys) {         // most often: nothing to look at
#pragma unroll
                    for (uint32_t run = 0; run < 2u; ++run) {
                        const uint8_t *kc = a.c.k_codes + at[run] * S::row + lane * 16u, *vc = a.c.v_codes + at[run] * S::row + lane * 16u;
#pragma unroll
                        for (uint32_t i = 0; i < pieces / 2; ++i) {
                            const uint32_t dst = st + swizzle<S::row>(((run * pieces / 2 + i) * 32u + lane) * 16u);
                            cp16_once(dst, kc + i * 512u, true, once);
                            cp16_once(dst + S::codes, vc + i * 512u, true, once);
                        }
                    }
                } else {
#pragma unroll 1
                    for (uint32_t i = 0; i < pieces; ++i) {
                        const uint32_t run = i * 2u >= pieces, p = i * 32u + lane - run * 16u * pieces;
                        const uint32_t r = run * 16u + p / pieces;
                        const uint64_t src = (run ? at[1] : at[0]) * S::row + p * 16u;
                        const uint32_t dst = st + swizzle<S::row>((i * 32u + lane) * 16u);
                        const bool ok = r < (run ? keys1 : keys0);
                        cp16_or_zero(dst, a.c.k_codes + (ok ? src : 0ull), ok);
                        cp16_or_zero(dst + S::codes, a.c.v_codes + (ok ? src : 0ull), ok);
                    }
                }
                // Scales: 16 bytes are 16 / blocks keys.
#pragma unroll
                for (uint32_t i = 0; i < (S::scales / 16 + 31) / 32; ++i) {
                    const uint32_t p = i * 32u + lane;
                    if (p < S::scales / 16) {
                        const uint32_t r = p * 16u / S::blocks, run = r >> 4;
                        const uint64_t src = (run ? at[1] : at[0]) * S::blocks + p * 16u - run * 16u * S::blocks;
                        const bool ok = r < (run ? keys1 : keys0);
                        cp16_or_zero(st + 2 * S::codes + p * 16u, a.c.k_scales + (ok ? src : 0ull), ok);
                        cp16_or_zero(st + 2 * S::codes + S::scales + p * 16u, a.c.v_scales + (ok ? src : 0ull), ok);
                    }
                }
            }
            cp_commit();
        };

        constexpr uint32_t stride = kWarps * kKeys;
        uint32_t key = k0 + warp * kKeys, slot = 0, page[2], ahead[2];
        look(key, page);
        look(key + stride, ahead);
        bool first_turn = true;
        if (key < k1)
            issue(key, 0, page);

        // Queries: f16 rows times their factors, a warp's rows at the same time.
        float *factor = &stat[0][0][0];
        {
            constexpr uint32_t per = D / 32, mine = kRows / kWarps;     // values of a lane, rows of a warp
            uint32_t x[mine][per / 2];
#pragma unroll
            for (uint32_t n = 0; n < mine; ++n) {
                const uint32_t row = tile * kRows + warp + n * kWarps, i = fastdiv(row, a.groupdiv), h = row - i * a.group;
                const uint16_t *src = a.q + (int64_t)(first + i) * a.q_stride + ((uint64_t)head * a.group + h) * D + lane * per;
#pragma unroll
                for (uint32_t j = 0; j < per / 2; ++j)
                    x[n][j] = row < rows ? __ldg(reinterpret_cast<const uint32_t *>(src) + j) : 0u;
            }
#pragma unroll
            for (uint32_t n = 0; n < mine; ++n) {
                const uint32_t r = warp + n * kWarps;
                uint32_t m = 0;
#pragma unroll
                for (uint32_t j = 0; j < per / 2; ++j)
                    m = absmax_bf16x2(m, x[n][j]);
                m = __reduce_max_sync(0xFFFFFFFFu, fold_halves(m)) << 16;
                const float f = row_factor(m);
#pragma unroll
                for (uint32_t j = 0; j < per / 2; ++j)
                    *reinterpret_cast<uint32_t *>(qs + r * S::q_pitch + (lane >> 3) * S::q_run + ((lane & 7u) * per + 2 * j) * 2) =
                        half2_bits(bf16_lo(x[n][j]) * f, bf16_hi(x[n][j]) * f);
                if (lane == 0)
                    factor[r] = 1.0f / f;
            }
        }
        __syncthreads();
        // Of this lane's rows 2 t4 and 2 t4 + 1 of every 8: log2-scale factor and last key.
        float fq[NT][2];
        int64_t pos[NT][2];     // rows past the sequence's see every key, and are not stored
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t r = nt * 8 + 2 * t4 + i, row = tile * kRows + r;
                fq[nt][i] = factor[r] * a.scale;
                pos[nt][i] = row < rows ? pos0 + fastdiv(row, a.groupdiv) : 0x7FFFFFFF;
            }
        // This lane's run of a query: values [t4 D / 4, + D / 4) of row g8 of every 8.
        uint4 q[NT][S::q_regs ? D / 32 : 1];        // of two products each
        const char *qa = qs + g8 * S::q_pitch + t4 * S::q_run;
        if (S::q_regs)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < D / 32; ++i)
                    q[nt][i] = lds128(qa + nt * 8 * S::q_pitch + i * 16);
        float kfac = 1.0f;
        if (FMT == MXQ_FMT_NVFP4)
            kfac = __ldg(a.c.k_s2 + head);

        float acc[D / 16][NT][4];
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                acc[j][nt][0] = acc[j][nt][1] = acc[j][nt][2] = acc[j][nt][3] = 0.0f;
        float mx[NT][2], sum[NT][2];        // references and sums
        ValueRef vref;                      // of the block of this lane's columns (MXFP8)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            mx[nt][0] = mx[nt][1] = kLowest;
            sum[nt][0] = sum[nt][1] = 0.0f;
        }

#pragma unroll 1
        for (; key < k1; key += stride, slot ^= 1u) {
            page[0] = ahead[0];
            page[1] = ahead[1];
            look(key + 2u * stride, ahead);
            issue(key + stride, slot ^ 1u, page);
            cp_wait<1>();
            __syncwarp();
            const char *st = ring + slot * S::stage;
            const char *ksc = st + 2 * S::codes, *vsc = ksc + S::scales;
            const uint32_t left = k1 - key;             // keys of the turn

            // Scores: 16 keys at a time, of which this lane decodes g8 and g8 + 8.
            float s[2][NT][4];
#pragma unroll
            for (uint32_t half = 0; half < 2u; ++half) {
                constexpr int nblk = S::fp4 ? D / 64 : (D + 127) / 128;         // blocks of the lane's run
                uint32_t kscale[2][nblk];               // f16x2
                float kf = kfac;
                const uint32_t kr = half * 16u + g8;
                if (S::fp4) {
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        const char *p = ksc + (kr + nt * 8) * S::blocks + t4 * (D / 64);
                        uint32_t w = 0;
                        if (D == 64)
                            w = *reinterpret_cast<const uint8_t *>(p);
                        else if (D == 128)
                            w = *reinterpret_cast<const uint16_t *>(p);
                        else
                            w = lds32(p);
                        if (kr + nt * 8 >= left)
                            w = 0u;
                        uint32_t h0, h1;
                        e4m3x4_unpack(w, h0, h1);
                        kscale[nt][0] = __byte_perm(h0, 0, 0x1010);
                        if (D >= 128)
                            kscale[nt][D >= 128 ? 1 : 0] = __byte_perm(h0, 0, 0x3232);
                        if (D == 256) {
                            kscale[nt][D == 256 ? 2 : 0] = __byte_perm(h1, 0, 0x1010);
                            kscale[nt][D == 256 ? 3 : 0] = __byte_perm(h1, 0, 0x3232);
                        }
                    }
                } else {
                    uint32_t e[2][nblk], top = kZeros;      // what is below counts as zeros (2^-100)
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                        for (int j = 0; j < nblk; ++j) {
                            const uint32_t blk = D == 64 ? t4 >> 1 : D == 128 ? t4 : t4 * 2 + j;
                            e[nt][j] = *reinterpret_cast<const uint8_t *>(ksc + (kr + nt * 8) * S::blocks + blk);
                            if (kr + nt * 8 >= left)
                                e[nt][j] = 0u;
                            top = max(top, e[nt][j]);
                        }
                    top = __reduce_max_sync(0xFFFFFFFFu, top);
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                        for (int j = 0; j < nblk; ++j) {
                            const float f = __uint_as_float((uint32_t)max((int)(e[nt][j] + 134u) - (int)top, 0) << 23);
                            kscale[nt][j] = half2_bits(f, f);
                        }
                    kf = __uint_as_float(top << 23) * 0x1p-7f;
                }
                float c[NT][4];
                constexpr int run = S::row / 4;          // bytes of a lane's run of a key
#pragma unroll
                for (int p = 0; p < (run + 15) / 16; ++p) {
                    uint32_t w[2][4];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const char *at = st + swizzle<S::row>((kr + n * 8) * S::row + t4 * run + p * 16);
                        if (run >= 16) {
                            const uint4 v = lds128(at);
                            w[n][0] = v.x, w[n][1] = v.y, w[n][2] = v.z, w[n][3] = v.w;
                        } else {
                            const uint2 v = lds64(at);
                            w[n][0] = v.x, w[n][1] = v.y;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < (run >= 16 ? 4 : 2); ++i) {
                        uint32_t h[2][4];
                        constexpr int per = S::fp4 ? 2 : 1;         // products of a word
#pragma unroll
                        for (int n = 0; n < 2; ++n)
                            if (S::fp4)
                                e2m1x8_unpack(w[n][i], h[n]);
                            else
                                e4m3x4_unpack(w[n][i], h[n][0], h[n][1]);
#pragma unroll
                        for (int u = 0; u < per; ++u) {
                            const int step = (p * 4 + i) * per + u;       // of 4 values of each lane
                            const int blk = S::fp4 ? step / 4 : step / 8;
                            const uint32_t a0 = hmul2_bits(h[0][2 * u], kscale[0][blk]), a2 = hmul2_bits(h[0][2 * u + 1], kscale[0][blk]);
                            const uint32_t a1 = hmul2_bits(h[1][2 * u], kscale[1][blk]), a3 = hmul2_bits(h[1][2 * u + 1], kscale[1][blk]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                if (!S::q_regs && step % 2 == 0)
                                    q[nt][0] = lds128(qa + nt * 8 * S::q_pitch + step * 8);
                                const uint4 x = q[nt][S::q_regs ? step / 2 : 0];
                                const uint32_t lo = step % 2 ? x.z : x.x, hi = step % 2 ? x.w : x.y;
                                if (step == 0)
                                    mma16816_first(c[nt], a0, a1, a2, a3, lo, hi);
                                else
                                    mma16816(c[nt], a0, a1, a2, a3, lo, hi);
                            }
                        }
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        // (rounded here, not with the subtraction below: no weight is above 2^kLag
                    // whatever the scores' size)
                    s[half][nt][j] = __fmul_rn(c[nt][j], fq[nt][j & 1] * kf);
            }

            // The largest scale of the values of this lane's block; lanes of a g8 have a quarter each.
            float shift = 1.0f;
            if (!S::fp4) {
                uint32_t vtop = 0u;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t r = (i >> 1) * 8 + 2 * t4 + (i & 1), blk = D == 64 ? g8 >> 2 : D == 128 ? g8 >> 1 : g8;
                    const uint32_t e = *reinterpret_cast<const uint8_t *>(vsc + r * S::blocks + blk);
                    vtop = max(vtop, r < left ? e : 0u);
                }
                vtop = max(vtop, __shfl_xor_sync(0xFFFFFFFFu, vtop, 1));
                vtop = max(vtop, __shfl_xor_sync(0xFFFFFFFFu, vtop, 2));
                shift = vref.follow(vtop, 1u);
            }

            // The reference (attention.cuh), and weights.
            int lim[NT][2], least = kKeys - 1;          // last key of the turn that a row sees
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    lim[nt][i] = (int)max(min(pos[nt][i] - (int64_t)key, (int64_t)min(left, kKeys) - 1), (int64_t)-1);
                    least = min(least, lim[nt][i]);
                }
            const bool cut = __any_sync(0xFFFFFFFFu, least < (int)kKeys - 1);
            float alpha[NT][2];
            bool moved = shift != 1.0f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float m = -INFINITY;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int j = i; j < 4; j += 2) {
                            if (cut)
                                s[h][nt][j] = (int)(h * 16 + (j >> 1) * 8 + g8) <= lim[nt][i] ? s[h][nt][j] : -INFINITY;
                            m = fmaxf(m, s[h][nt][j]);
                        }
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1)
                        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                    alpha[nt][i] = 1.0f;
                    if (m - mx[nt][i] > kLag) {         // the weights' own difference, rounded as theirs
                        m -= kTop;
                        alpha[nt][i] = ex2(mx[nt][i] - m);
                        mx[nt][i] = m;
                        moved = true;
                    }
                    float part = 0.0f;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int j = i; j < 4; j += 2) {
                            s[h][nt][j] = ex2(s[h][nt][j] - mx[nt][i]);
                            part += s[h][nt][j];
                        }
                    sum[nt][i] = fmaf(sum[nt][i], alpha[nt][i], part);
                }
            if (!first_turn && __any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        acc[j][nt][0] *= alpha[nt][0] * shift;
                        acc[j][nt][1] *= alpha[nt][1] * shift;
                        acc[j][nt][2] *= alpha[nt][0] * shift;
                        acc[j][nt][3] *= alpha[nt][1] * shift;
                    }
            }
            first_turn = false;
            // A lane has a key's weights for two rows; the products want a row's for two keys.
            uint32_t pw[2][NT][2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    pw[h][nt][0] = transpose8(half2_bits(s[h][nt][0], s[h][nt][1]));
                    pw[h][nt][1] = transpose8(half2_bits(s[h][nt][2], s[h][nt][3]));
                }

            // Outputs: 16 keys at a time, columns d = run of this lane.
#pragma unroll
            for (uint32_t kk = 0; kk < 2u; ++kk) {
                constexpr int vblocks = S::fp4 && D == 256 ? 2 : 1;      // of a lane's run of D / 8
                uint32_t vscale[2][vblocks];        // of the key pairs 2 t4, + 1 and 8 further
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < vblocks; ++j) {
                        const uint32_t r = kk * 16u + i * 8 + 2 * t4;
                        const uint32_t blk = S::fp4 ? (D == 64 ? g8 >> 1 : D == 128 ? g8 : g8 * 2 + j)
                                                    : (D == 64 ? g8 >> 2 : D == 128 ? g8 >> 1 : g8);
                        uint32_t w0 = *reinterpret_cast<const uint8_t *>(vsc + r * S::blocks + blk);
                        uint32_t w1 = *reinterpret_cast<const uint8_t *>(vsc + (r + 1) * S::blocks + blk);
                        w0 = r < left ? w0 : 0u;
                        w1 = r + 1 < left ? w1 : 0u;
                        if (S::fp4)
                            vscale[i][j] = e4m3x2_to_f16x2(w0 | (w1 << 8));
                        else
                            vscale[i][j] = half2_bits(__uint_as_float((uint32_t)max((int)(w0 + 134u) - (int)vref.ref, 0) << 23),
                                                      __uint_as_float((uint32_t)max((int)(w1 + 134u) - (int)vref.ref, 0) << 23));
                    }
                constexpr int run = S::row / 8;          // bytes of a lane's run of columns
                constexpr int words = run < 16 ? run / 4 : 4;
                const char *vs = st + S::codes;
#pragma unroll
                for (int p = 0; p < (run + 15) / 16; ++p) {
                    uint32_t w[4][words];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t r = kk * 16u + (i >> 1) * 8 + 2 * t4 + (i & 1);
                        // of two pieces the lanes of odd g8 take the second first (banks)
                        const uint32_t off = r * S::row + g8 * run + (run == 32 ? (p ^ (g8 & 1u)) * 16u : 0u);
                        const char *q = vs + swizzle<S::row>(off);
                        if (words == 4) {
                            const uint4 v = lds128(q);
                            w[i][0] = v.x, w[i][words > 1 ? 1 : 0] = v.y, w[i][words > 2 ? 2 : 0] = v.z, w[i][words > 2 ? 3 : 0] = v.w;
                        } else if (words == 2) {
                            const uint2 v = lds64(q);
                            w[i][0] = v.x, w[i][words > 1 ? 1 : 0] = v.y;
                        } else
                            w[i][0] = lds32(q);
                    }
#pragma unroll
                    for (int i = 0; i < words; ++i) {
                        if (S::fp4) {
                            // nibbles of two keys side by side: codes 0, 2, 4, 6 and 1, 3, 5, 7 of the word
                            const uint32_t lm = 0x0F0F0F0Fu;
                            uint32_t b0[2][4], b1[2][4];
                            e2m1x8_unpack((w[0][i] & lm) | ((w[1][i] << 4) & ~lm), b0[0]);
                            e2m1x8_unpack(((w[0][i] >> 4) & lm) | (w[1][i] & ~lm), b0[1]);
                            e2m1x8_unpack((w[2][i] & lm) | ((w[3][i] << 4) & ~lm), b1[0]);
                            e2m1x8_unpack(((w[2][i] >> 4) & lm) | (w[3][i] & ~lm), b1[1]);
                            const int blk = vblocks == 2 ? i / 2 : 0;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t a0 = hmul2_bits(b0[0][j], vscale[0][blk]), a1 = hmul2_bits(b0[1][j], vscale[0][blk]);
                                const uint32_t a2 = hmul2_bits(b1[0][j], vscale[1][blk]), a3 = hmul2_bits(b1[1][j], vscale[1][blk]);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    mma16816(acc[(p * words + i) * 4 + j][nt], a0, a1, a2, a3, pw[kk][nt][0], pw[kk][nt][1]);
                            }
                        } else {
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                uint32_t x0, x1, y0, y1;
                                e4m3x4_unpack(__byte_perm(w[0][i], w[1][i], u ? 0x7362 : 0x5140), x0, x1);
                                e4m3x4_unpack(__byte_perm(w[2][i], w[3][i], u ? 0x7362 : 0x5140), y0, y1);
                                const uint32_t a0 = hmul2_bits(x0, vscale[0][0]), a1 = hmul2_bits(x1, vscale[0][0]);
                                const uint32_t a2 = hmul2_bits(y0, vscale[1][0]), a3 = hmul2_bits(y1, vscale[1][0]);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    mma16816(acc[(p * words + i) * 2 + u][nt], a0, a1, a2, a3, pw[kk][nt][0], pw[kk][nt][1]);
                            }
                        }
                    }
                }
            }
            __syncwarp();
        }
        cp_wait<0>();

        // Join the warps: sums over the lanes of a row first.
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int o = 4; o < 32; o <<= 1)
                    sum[nt][i] += __shfl_xor_sync(0xFFFFFFFFu, sum[nt][i], o);
        __syncthreads();
        if (g8 == 0)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    stat[0][warp][nt * 8 + 2 * t4 + i] = mx[nt][i];
                    stat[1][warp][nt * 8 + 2 * t4 + i] = sum[nt][i];
                }
        __syncthreads();
        float *outs = reinterpret_cast<float *>(smem) + warp * (S::outs / 4);
        // Row r's reference and sum of all warps.
        auto row_stat = [&](uint32_t r, float &l) {
            float m = stat[0][0][r];
#pragma unroll
            for (uint32_t w = 1; w < kWarps; ++w)
                m = fmaxf(m, stat[0][w][r]);
            l = 0.0f;
#pragma unroll
            for (uint32_t w = 0; w < kWarps; ++w)
                l = fmaf(stat[1][w][r], ex2(stat[0][w][r] - m), l);
            return m;
        };
        // Each warp's share of the CTA's output: divided by the sum here, so that values near the
        // end of fp32's range stay in it.
        const float unit = S::fp4 ? 1.0f : vref.unit();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t r = nt * 8 + 2 * t4 + i;
                float l;
                const float m = row_stat(r, l), f = ex2(mx[nt][i] - m) * inverse(l);
                // the run of lanes g8, two values a product
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    const uint32_t jj = S::row == 256 ? (2 * j) ^ ((g8 & 1u) * 16u) : 2 * j;
                    *reinterpret_cast<float2 *>(outs + r * (D + 4) + g8 * (D / 8) + jj) =
                        make_float2(acc[j][nt][i] * f * unit, acc[j][nt][2 + i] * f * unit);
                }
            }
        __syncthreads();
        const float vfac = FMT == MXQ_FMT_NVFP4 ? __ldg(a.c.v_s2 + head) : 1.0f;
        const bool whole = walk.whole();
        float *part = part_of<kRows, D>(a, blockIdx.x, walk.slot());
        auto put = [&](uint32_t r, uint32_t d, float m, float l, float4 v) {        // 4 columns of a finished row; m, l where d is 0
            const uint32_t row = tile * kRows + r, it = fastdiv(row, a.groupdiv), h = head * a.group + row - it * a.group;
            const uint64_t out = (uint64_t)(first + it) * (a.c.heads * a.group) + h;
            const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * vfac, v.y * vfac), hi = __floats2bfloat162_rn(v.z * vfac, v.w * vfac);
            *reinterpret_cast<uint2 *>(a.o + out * D + d) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
            if (d == 0 && a.lse)
                a.lse[out] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
        };
        if (!CLUSTER && walk.earlier())
            add_earlier<kRows, D, S::outs / 4>(reinterpret_cast<float *>(smem), &stat[0][0][0], part);
        const float *all = reinterpret_cast<const float *>(smem);
        float *sum4 = reinterpret_cast<float *>(smem);      // CLUSTER: the CTA's outputs, over the first warp's
#pragma unroll 1
        for (uint32_t i = tid; i < kRows * (D / 4); i += kThreads) {
            const uint32_t r = i / (D / 4), d = i % (D / 4) * 4;
            if (tile * kRows + r >= rows)
                continue;
            float m = 0.0f, l = 0.0f;
            if (d == 0)
                m = row_stat(r, l);
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (uint32_t w = 0; w < kWarps; ++w) {
                const float4 x = *reinterpret_cast<const float4 *>(all + w * (S::outs / 4) + r * (D + 4) + d);
                v.x += x.x;
                v.y += x.y;
                v.z += x.z;
                v.w += x.w;
            }
            if (CLUSTER && ranks > 1u) {
                *reinterpret_cast<float4 *>(sum4 + r * (D + 4) + d) = v;        // read by this thread alone
                if (d == 0) {
                    joint[0][r] = m;
                    joint[1][r] = l;
                }
            } else if (CLUSTER || whole)
                put(r, d, m, l, v);
            else {
                *reinterpret_cast<float4 *>(part + r * D + d) = v;
                if (d == 0)
                    *reinterpret_cast<float2 *>(part + kRows * D + r * 2) = make_float2(m, l);
            }
        }
        if (CLUSTER && ranks > 1u) {
            cluster_sync_all();
            // Each CTA joins its share of the columns, in the order of the CTAs.
#pragma unroll 1
            for (uint32_t i = rank * kThreads + tid; i < kRows * (D / 4); i += ranks * kThreads) {
                const uint32_t r = i / (D / 4), d = i % (D / 4) * 4;
                if (tile * kRows + r >= rows)
                    continue;
                float share[8], m = kLowest, l = 0.0f;      // of the CTAs (8 at most)
#pragma unroll
                for (uint32_t c = 0; c < 8u; ++c) {
                    share[c] = c < ranks ? peer_f(&joint[0][r], c) : kLowest;
                    m = fmaxf(m, share[c]);
                }
#pragma unroll
                for (uint32_t c = 0; c < 8u; ++c)
                    if (c < ranks) {
                        share[c] = peer_f(&joint[1][r], c) * ex2(share[c] - m);
                        l += share[c];
                    }
                const float f = inverse(l);
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (uint32_t c = 0; c < 8u; ++c)
                    if (c < ranks) {
                        const float4 x = peer_f4(reinterpret_cast<const float4 *>(sum4 + r * (D + 4) + d), c);
                        const float g = share[c] * f;
                        v.x = fmaf(x.x, g, v.x);
                        v.y = fmaf(x.y, g, v.y);
                        v.z = fmaf(x.z, g, v.z);
                        v.w = fmaf(x.w, g, v.w);
                    }
                put(r, d, m, l, v);
            }
            cluster_sync_all();         // every CTA's sums have been read
        }
        if (!CLUSTER && tid == 0 && walk.unfinished()) {
            Unfinished u = {};
            u.first = first;
            u.row0 = tile * kRows;
            u.rows = rows;
            u.head = head;
            u.parts = parts_of(range, walk.steps, walk.k1);
            a.left[blockIdx.x] = u;
        }
        __syncthreads();
    }
}

namespace {

template <int FMT, int D, int NT>
cudaError_t run(const AttArgs &a, uint32_t sms, uint32_t &ctas, cudaStream_t s)
{
    using S = Shape<FMT, D, NT>;
    const auto k = attention_rows_kernel<FMT, D, NT, false>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::all);
    ctas = sms * S::fit;
    return e != cudaSuccess ? e : launch_dependent(k, dim3(ctas), 32 * kWarps, S::all, s, a);
}

// Clusters of 1 to 8 CTAs, one a tile, where they fit the card at once.  most_keys: what a
// sequence can have.
template <int FMT, int D, int NT>
cudaError_t run_clusters(const AttArgs &a, uint32_t sms, uint64_t most_keys, bool &taken, cudaStream_t s)
{
    using S = Shape<FMT, D, NT>;
    const uint64_t clusters = (uint64_t)a.c.seqs * a.c.heads * a.tiles, room = (uint64_t)sms * S::fit;
    uint32_t size = 1;
    while (size < 8u && clusters * size * 2u <= room && (uint64_t)size * kWarps * kKeys < most_keys)
        size *= 2u;
    // turns of a warp, at most: beyond these the work is divided evenly
    taken = clusters <= room && most_keys <= (uint64_t)size * kWarps * kKeys * kClusterTurns;
    if (!taken)
        return cudaSuccess;
    const auto k = attention_rows_kernel<FMT, D, NT, true>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::all);
    if (e != cudaSuccess)
        return e;
    const dim3 grid((unsigned)(clusters * size));
    return size == 1   ? launch_dependent<1>(k, grid, 32 * kWarps, S::all, s, a)
           : size == 2 ? launch_dependent<2>(k, grid, 32 * kWarps, S::all, s, a)
           : size == 4 ? launch_dependent<4>(k, grid, 32 * kWarps, S::all, s, a)
                       : launch_dependent<8>(k, grid, 32 * kWarps, S::all, s, a);
}

template <int FMT, int D, int NT>
cudaError_t either(const AttArgs &a, uint32_t sms, uint64_t most_keys, uint32_t &ctas, cudaStream_t s)
{
    bool taken = false;
    ctas = 0;
    const cudaError_t e = run_clusters<FMT, D, NT>(a, sms, most_keys, taken, s);
    return taken || e != cudaSuccess ? e : run<FMT, D, NT>(a, sms, ctas, s);
}

} // namespace

// `ctas`: of a launch that leaves unfinished tiles, each with its entry in `left`; 0 of
// one that does not.  Tiles of `rows` rows, 8 or 16.
template <int FMT, int D>
static cudaError_t sized(const AttArgs &a, uint32_t rows, uint32_t sms, uint64_t most_keys, uint32_t &ctas, cudaStream_t s)
{
    return rows == 8u ? either<FMT, D, 1>(a, sms, most_keys, ctas, s) : either<FMT, D, 2>(a, sms, most_keys, ctas, s);
}

cudaError_t launch_attention_rows(const AttArgs &a, int fmt, int dim, uint32_t rows, uint32_t sms, uint64_t most_keys,
                                  uint32_t &ctas, cudaStream_t s)
{
    if (fmt == MXQ_FMT_NVFP4)
        return dim == 64    ? sized<MXQ_FMT_NVFP4, 64>(a, rows, sms, most_keys, ctas, s)
               : dim == 128 ? sized<MXQ_FMT_NVFP4, 128>(a, rows, sms, most_keys, ctas, s)
                            : sized<MXQ_FMT_NVFP4, 256>(a, rows, sms, most_keys, ctas, s);
    return dim == 64    ? sized<MXQ_FMT_MXFP8, 64>(a, rows, sms, most_keys, ctas, s)
           : dim == 128 ? sized<MXQ_FMT_MXFP8, 128>(a, rows, sms, most_keys, ctas, s)
                        : sized<MXQ_FMT_MXFP8, 256>(a, rows, sms, most_keys, ctas, s);
}

} // namespace mxq
