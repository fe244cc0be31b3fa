// attention_tiles.cu -- attention over a quantized cache where a sequence has many
// rows: chunks of a prompt (sm_100a).  The products are the work.
//
// A tile is 256 rows (128 for heads of 256 values) of one sequence and key/value
// head, a step 64 keys; attention.cuh divides them among one CTA an SM.  Both products
// run on tcgen05: S = Q K^T from shared memory into TMEM, O += P V with P from TMEM.
// Warps 8-10 decode the keys' codes straight from global memory into f16 tiles in
// shared memory, warps 12-14 the values' (four stages each, two for heads of 256; the
// same layout for both: rows of a token, 128 bytes wide, 128-byte swizzle; the values' is
// read as an MN-major operand, so nothing is transposed).  Warps 0-3 and 4-7 are two
// groups that take the softmax of 128 rows each, a row a thread, so a row's maximum and
// sum need no exchange; while one works the tensor cores do the other's products.  Warps
// 11 and 15 issue, one for each group.
//
// Scores lie in four TMEM buffers of 64 columns, whose first halves take the weights.
// With two groups at work each has two of them, with one (tiles of up to 128 rows) it has
// all four; scores of a step are issued as soon as the product that reads the weights in
// their place is done, a buffer's count of steps ahead.
//
// Weights are taken against a reference (attention.cuh); only where a score lies too far
// above it is the maximum found, the step's weights are taken again, and the output
// in TMEM is rescaled (by the softmax group, which has the output to itself between its
// products).  MXFP8 powers: keys as in attention_rows.cu, a largest one for every 32 (16) keys.
// Values are relative to a reference of the step (ValueRef), which may stand 2^4 above its largest
// scale (exact within 2^18 then).  The warps that decode keys, ahead of the others, tell the
// largest scales of the values of their chunks (heads of 256, whose decoding is what a step waits
// for: warp 15 does, 976 us for 2048 tokens over 10240 otherwise); those that decode values follow
// them step by step, so that all use the same, and the softmax has no more to do than rescale
// the output where it moved.
//
// Bound: a step of 256 x 64 x 128 costs the tensor cores 1024 cycles and the SM's 16
// exponentials a cycle 1024 as well, beside which a softmax thread has two operations a
// score in fp32 and a rounding to f16.  A chunk of 4096 tokens over 20480 of 32 query and
// 4 key/value heads of 128 takes 1.35 ms (916 TFLOP/s, 56 % of the measured rate of a
// bf16 product; NVFP4 1.28 ms; heads of 64 1.25 ms, of 256 half the chunk over 10240
// 0.91 ms).  Each is busy for 42 to 44 % of that: a step takes 2500 cycles, in a group's
// chain from scores to weights and products issued one behind the other.  Steps that
// brought it there: 2.46 ms with one warp that issued for all and steps of 128 keys; 1.71
// with products issued by the groups; 1.54 with steps of 64 keys and an issuing warp a group
// (a warp is held while its products queue); 1.49 with fewer waits between weights and
// scores; 1.26 with one copy of each loop and the division of the work out of line (a launch
// begins with cold instruction caches); scores rounded before the reference is subtracted
// and references of the values brought it back to 1.35.  A polynomial in place of part of the
// exponentials, other shares of registers, and softmax threads that share a row were slower
// or no faster.
//
// Every wait is bounded (MXQ_DEV_WAIT_TIMEOUT); all roles then leave, the issuing
// ones behind their last product.
#include "attention.cuh"
#include "mxq_mma.cuh"
#include "mxq_tcgen05.cuh"
#include "mxq_test.h"
#include <algorithm>
#include <atomic>

namespace mxq {

namespace {

// Test hook (include/mxq_test.h): the next launch stalls on purpose.
std::atomic<int> g_stall_attention{0};

// Tests of a barrier before a wait gives up.  A test suspends for 4 us at most, so that is
// after a second; a step takes microseconds.  A group that has nothing to do waits for the
// other's whole tiles, 8 times as long (and leaves at once where the other gives up).
// (In a launch that was told to stall a sixteenth of that.)
constexpr uint32_t kSpin = 1u << 18, kStalledSpin = 1u << 14, kIdle = 8;
constexpr uint32_t kCodeWarp = 8;
constexpr uint32_t kMostSteps = 512;        // of a piece: 2^15 keys
constexpr int kThreads = 512;

template <int FMT, int D>
struct Shape {
    static constexpr bool fp4 = FMT == MXQ_FMT_NVFP4;
    static constexpr uint32_t row = fp4 ? D / 2 : D;            // bytes of a token's codes
    static constexpr uint32_t blocks = fp4 ? D / 16 : D / 32;   // and of its scales
    static constexpr uint32_t log = 6, keys = 1u << log;        // of a step
    static constexpr uint32_t mine = D == 256 ? 16 : 32;        // keys of a chunk, one turn of a decoding warp
    static constexpr uint32_t chunks = keys / mine;
    static constexpr uint32_t subs = D == 256 ? 1 : 2, rows = 128 * subs;
    static constexpr uint32_t panel = keys * 128;               // 64 values of a step's tokens
    static constexpr uint32_t qpanel = 128 * 128;
    static constexpr uint32_t qbytes = 128 * D * 2, tile = keys * D * 2;
    static constexpr uint32_t stages = D == 256 ? 2 : 4;        // of keys, and of values
    static constexpr uint32_t smem = subs * qbytes + 2 * stages * tile + 1024;
    static constexpr uint32_t pieces = row / 16;                // of a token's codes
    static constexpr uint32_t loads = mine * pieces / 32;       // pieces of a lane
};

constexpr uint32_t kBufs = 4;               // of scores, in TMEM
constexpr uint32_t kRing = 16;              // steps whose powers are kept; decoding is fewer ahead
struct Bars {
    uint64_t kfull[4], kempty[4], vfull[4], vempty[4], sfull[kBufs], pfull[kBufs], pv[2], odone[2], qfull[2], ffull[kRing];
    uint64_t tfull[kRing], tempty[kRing], meet, drain[2];
    uint32_t tmem, abort;
    float kfac[kRing][4];       // by step and chunk: powers of the keys,
    uint32_t vtop[kRing];       // by step: largest scales of the values, a byte a chunk
    uint32_t vref[kRing];       // and what they are relative to
};

// Further tests of a barrier whose first one failed.
__device__ __noinline__ bool wait_more(uint64_t *bar, uint32_t parity, Bars &s, uint32_t *status, uint32_t spin)
{
    for (uint32_t i = 0; i < spin; ++i) {
        if (mbar_try_wait(bar, parity))
            return true;
        if ((i & 63u) == 63u && *reinterpret_cast<volatile uint32_t *>(&s.abort))
            return false;
    }
    *reinterpret_cast<volatile uint32_t *>(&s.abort) = 1u;
    atomicOr(status, MXQ_DEV_WAIT_TIMEOUT);
    return false;
}
// The whole warp.
__device__ __forceinline__ bool wait_all(uint64_t *bar, uint32_t parity, Bars &s, const AttArgs &a, uint32_t times = 1)
{
    return __all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity & 1u)) ||
           __all_sync(0xFFFFFFFFu, wait_more(bar, parity & 1u, s, a.c.status, a.spin * times));
}

// 128 x N products of 16, f16 operands, from shared memory and from TMEM; issued
// by the lane whose `one` is 1.
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add, uint32_t one)
{
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "setp.ne.u32 p, %4, 0;\n\t"
                 "setp.ne.u32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"(one) : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add, uint32_t one)
{
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "setp.ne.u32 p, %4, 0;\n\t"
                 "setp.ne.u32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"(one) : "memory");
}

// Descriptor of an MN-major operand: rows (of the products' K) of 128 bytes, the
// 128-byte swizzle, 8 rows 1024 bytes apart and 64 columns `panel` bytes apart.
__device__ __forceinline__ uint64_t columns_desc(uint32_t addr, uint32_t panel)
{
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(panel >> 4) << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// 16 columns of this warp's 32 TMEM lanes, one lane a thread.
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&v)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
                 "%13, %14, %15, %16};"
                 ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
                   "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]) : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&v)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
                 "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
                 ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
                   "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
                   "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]),
                   "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31]) : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// What the pieces of a tile before this one left of this thread's row is added to its output in
// TMEM, which is then that of all of them, and no sum any more; their reference and sum.
template <int D>
__device__ __noinline__ float2 add_earlier(uint32_t out, const float4 *row, const float2 *stat, float mx, float sum, float unit)
{
    const float2 st = *stat;
    const float top = fmaxf(st.x, mx), share = st.y * ex2(st.x - top), own = ex2(mx - top), all = fmaf(sum, own, share);
    const float f = own * inverse(all), g = share * inverse(all);
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(out + c * 32, o);
        tmem_ld_wait(o);
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const float4 e = row[c * 8 + x];
            o[x * 4] = __float_as_uint(fmaf(e.x, g, __uint_as_float(o[x * 4]) * f * unit));
            o[x * 4 + 1] = __float_as_uint(fmaf(e.y, g, __uint_as_float(o[x * 4 + 1]) * f * unit));
            o[x * 4 + 2] = __float_as_uint(fmaf(e.z, g, __uint_as_float(o[x * 4 + 2]) * f * unit));
            o[x * 4 + 3] = __float_as_uint(fmaf(e.w, g, __uint_as_float(o[x * 4 + 3]) * f * unit));
        }
        tmem_st32(out + c * 32, o);
    }
    tmem_st_wait();
    return make_float2(top, all);
}

// How the units of a piece lie: `two` groups, or the first alone.
template <typename S>
struct Units {
    bool two;
    uint32_t steps, all;
    template <typename W>
    __device__ __forceinline__ Units(const W &w)
        : two(S::subs == 2 && min(w.s.rows - w.rt * S::rows, S::rows) > 128u), steps(w.k1 - w.k0),
          all(two ? 2u * steps : steps) {}
    // TMEM buffer of group g's step j, the number of that use, and the uses of buffer i in all.
    __device__ __forceinline__ uint32_t buffer(uint32_t g, uint32_t j) const { return (two ? 2u * j + g : j) % kBufs; }
    __device__ __forceinline__ uint32_t use(uint32_t j) const { return two ? j >> 1 : j >> 2; }
    __device__ __forceinline__ uint32_t uses(uint32_t i) const { return (all + kBufs - 1u - i) / kBufs; }
    // Products with the values of group i.
    __device__ __forceinline__ uint32_t products(uint32_t i) const { return two || i == 0 ? steps : 0u; }
};

// A decoding warp's part of a step: pieces of codes and their scales, in registers.
template <int FMT, int D>
struct Raw {
    using S = Shape<FMT, D>;
    uint4 c[S::loads];
    // NVFP4: the two scales of each piece.  MXFP8: the scales of key lane % mine.
    uint32_t s[S::fp4 ? S::loads : (S::blocks + 3) / 4];
    uint32_t v[S::fp4 || S::subs == 1 ? 1 : (S::blocks + 3) / 4];       // MXFP8, of a warp of keys: the scales of the same token's values
};

} // namespace

template <int FMT, int D>
__global__ void __launch_bounds__(kThreads, 1)
attention_tiles_kernel(const __grid_constant__ AttArgs a)
{
    using S = Shape<FMT, D>;
    using W = Walk<S::rows, S::log, kMostSteps>;
    extern __shared__ __align__(1024) char smem_raw[];
    __shared__ Bars bars;
    __shared__ Range range;
    __shared__ AttArgs sa;      // for functions out of line
    __shared__ W walks[16];     // of the warps
    char *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    char *kt = smem + S::subs * S::qbytes, *vt = kt + S::stages * S::tile;
    const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31u;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bars.kfull[i], S::chunks);
            mbar_init(&bars.kempty[i], S::subs);
            mbar_init(&bars.vfull[i], S::chunks);
            mbar_init(&bars.vempty[i], S::subs);
            mbar_init(&bars.sfull[i], 1);
            mbar_init(&bars.pfull[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.pv[i], 1);
            mbar_init(&bars.odone[i], 1);
            mbar_init(&bars.qfull[i], 4);
            mbar_init(&bars.drain[i], 1);
        }
        for (uint32_t i = 0; i < kRing; ++i) {
            mbar_init(&bars.ffull[i], 2 * S::chunks);
            mbar_init(&bars.tfull[i], S::subs == 2 ? S::chunks : 1);
            mbar_init(&bars.tempty[i], 3);
            bars.vtop[i] = 0;
        }
        mbar_init(&bars.meet, 8);
        bars.abort = 0;
        sa = a;
        fence_mbar_init();
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_addr(&bars.tmem)), "n"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();
    __syncthreads();
    find_range<typename W::Div>(sa, range);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = bars.tmem;
    if (threadIdx.x == 0)
        a.left[blockIdx.x].parts = 0u;
    // TMEM columns: scores in four buffers, whose first halves take the weights, and outputs.
    constexpr uint32_t kOut = kBufs * S::keys;
    static_assert(kOut + S::subs * D <= 512, "TMEM");

    // Largest of the warp's bytes.
    auto largest = [](uint32_t m) {
        m = __vmaxu4(m, m >> 16);
        return __reduce_max_sync(0xFFFFFFFFu, max(kZeros, max(m & 0xFFu, (m >> 8) & 0xFFu)));
    };

    W &w = walks[warp];
    if (!S::fp4 && S::subs == 1 && warp == kCodeWarp + 7u) {        // tells the largest scales of the values
        bool more = W::begin(w, sa, range);
        uint32_t step = w.k0, t = 0;
        uint2 s[2];
        auto load = [&]() {
#pragma unroll
            for (uint32_t i = 0; i < 2; ++i) {
                const uint32_t key = (step << S::log) + lane + 32u * i;
                const uint32_t page = key < w.keys ? table_entry(a.c, w.b, key) : a.c.pages;
                const uint64_t at = (((uint64_t)page * a.c.heads + w.head) << a.c.page_log) + (key & ((1u << a.c.page_log) - 1u));
                s[i] = page < a.c.pages ? __ldg(reinterpret_cast<const uint2 *>(a.c.v_scales + at * S::blocks)) : make_uint2(0u, 0u);
            }
        };
        if (more)
            load();
        for (; more; ++t) {
            const uint32_t m = __vmaxu4(__vmaxu4(s[0].x, s[0].y), __vmaxu4(s[1].x, s[1].y));
            if (++step == w.k1) {
                more = W::next(w, sa);
                step = w.k0;
            }
            if (more)
                load();
            const uint32_t top = largest(m);
            if (!wait_all(&bars.tempty[t % kRing], t / kRing + 1u, bars, a))        // (a fresh barrier passes)
                break;
            if (lane == 0) {
                bars.vtop[t % kRing] = top;
                mbar_arrive(&bars.tfull[t % kRing]);
            }
        }
    } else if (warp >= kCodeWarp && (warp & 3u) == 3u) {    // issue
        const uint32_t one = elect_one(), wg = (warp - kCodeWarp) >> 2;
        uint32_t t0 = 0, buf0[kBufs] = {0, 0, 0, 0}, q0 = 0, pv0 = 0;
        bool ok = wg < S::subs;
        constexpr uint32_t sdesc = (1u << 4) | ((S::keys / 8u) << 17) | (8u << 24);
        constexpr uint32_t odesc = (1u << 4) | (1u << 16) | ((D / 8u) << 17) | (8u << 24);
        const uint64_t qd = operand_desc(smem_addr(smem + wg * S::qbytes)), kd = operand_desc(smem_addr(kt));
        const uint64_t vd = columns_desc(smem_addr(vt), S::panel);
        const uint32_t out = tmem + kOut + wg * D;
        for (bool more = W::begin(w, sa, range); more && ok; more = W::next(w, sa)) {
            const Units<S> un(w);
            if (wg == 0u || un.two) {
                const uint32_t buffers = un.two ? kBufs / 2u : kBufs;       // of this group
                ok = wait_all(&bars.qfull[wg], q0++, bars, a, kIdle);
                auto keys_there = [&](uint32_t j) {
                    const uint32_t t = t0 + j;
                    ok = ok && wait_all(&bars.kfull[t % S::stages], t / S::stages, bars, a);
                };
                // Scores of step j; a group alone makes up for the other's arrivals.
                auto scores = [&](uint32_t j) {
                    const uint32_t t = t0 + j, stage = t % S::stages, buf = un.buffer(wg, j);
                    if (!ok)
                        return;
                    fence_after();
                    const uint64_t k1 = kd + stage * (S::tile >> 4);
#pragma unroll
                    for (uint32_t k = 0; k < D / 16; ++k)
                        umma_ss(tmem + buf * S::keys, qd + (k >> 2) * (S::qpanel >> 4) + (k & 3u) * 2u,
                                k1 + (k >> 2) * (S::panel >> 4) + (k & 3u) * 2u, sdesc, k > 0, one);
                    umma_commit(&bars.sfull[buf], one);
                    umma_commit(&bars.kempty[stage], one);
                    if (S::subs == 2 && !un.two)
                        umma_commit(&bars.kempty[stage], one);
                };
                for (uint32_t j = 0; j < min(un.steps, buffers); ++j) {
                    keys_there(j);
                    scores(j);
                }
                for (uint32_t j = 0; j < un.steps && ok; ++j) {
                    const uint32_t t = t0 + j, stage = t % S::stages, buf = un.buffer(wg, j);
                    if (j + buffers < un.steps)
                        keys_there(j + buffers);
                    ok = ok && wait_all(&bars.vfull[stage], t / S::stages, bars, a) &&
                         wait_all(&bars.pfull[buf], buf0[buf] + un.use(j), bars, a);
                    if (!ok)
                        break;
                    fence_after();
                    const uint64_t v1 = vd + stage * (S::tile >> 4);
#pragma unroll
                    for (uint32_t k = 0; k < S::keys / 16; ++k)
                        umma_ts(out, tmem + buf * S::keys + k * 8u, v1 + k * 128u, odesc, j > 0 || k > 0, one);
                    umma_commit(&bars.pv[wg], one);
                    umma_commit(&bars.vempty[stage], one);
                    if (S::subs == 2 && !un.two)
                        umma_commit(&bars.vempty[stage], one);
                    if (j + 1u == un.steps)
                        umma_commit(&bars.odone[wg], one);
                    // The weights have been read, and the next scores may take their place.
                    ok = wait_all(&bars.pv[wg], pv0 + j, bars, a);
                    if (j + buffers < un.steps)
                        scores(j + buffers);
                }
            }
            t0 += un.steps;
#pragma unroll
            for (uint32_t i = 0; i < kBufs; ++i)
                buf0[i] += un.uses(i);
            pv0 += un.products(wg);
        }
        umma_commit(&bars.drain[wg], one);           // every product of this warp is done
        for (uint32_t i = 0; i < kSpin && !mbar_try_wait(&bars.drain[wg], 0); ++i)
            ;
    } else if (warp >= kCodeWarp) {                  // decoding
        // Three warps take the chunks of keys in turn, three those of values.
        const bool values = warp >= kCodeWarp + 4u;
        constexpr uint32_t stride = 3;
        uint32_t dw = (warp & 3u) + S::chunks;
        const uint8_t *codes = values ? a.c.v_codes : a.c.k_codes, *scales = values ? a.c.v_scales : a.c.k_scales;
        uint64_t *full = values ? bars.vfull : bars.kfull, *empty = values ? bars.vempty : bars.kempty;
        char *tiles = values ? vt : kt;
        Raw<FMT, D> raw;
        bool more = W::begin(w, sa, range);
        uint32_t step = w.k0 - 1u, t = 0u - 1u;     // before the first
        // Steps that the warp passes on its way from a chunk to its next.
        constexpr uint32_t kPass = S::chunks == 2 ? 2 : 1;
        struct Passed {
            bool on, first;         // it is one; the first of a piece
            uint32_t t;
        } passed[kPass];
        ValueRef vref;
        auto settle = [&]() {       // the chunk is number dw from step `step` on: its own step
#pragma unroll
            for (uint32_t n = 0; n < kPass; ++n) {
                passed[n].on = dw >= S::chunks && more;
                if (!passed[n].on)
                    continue;
                dw -= S::chunks;
                if (++step == w.k1) {
                    more = W::next(w, sa);
                    step = w.k0;
                }
                passed[n].t = ++t;
                passed[n].first = step == w.k0;
            }
        };
        if (more)
            settle();
        // The lane's piece and row of a load, so that the 8 lanes of a store to shared memory
        // have pieces of one panel: 4 of 2 rows (E2M1, whose pieces are twice as long in f16,
        // 2 of 4), which the swizzle spreads over all banks.
        constexpr uint32_t low = S::fp4 ? 1u : 2u, mid = 3u - low;       // bits of the piece, of the row
        constexpr uint32_t bits = S::pieces == 2 ? 1u : S::pieces == 4 ? 2u : S::pieces == 8 ? 3u : 4u;
        const uint32_t piece0 = (lane & ((1u << low) - 1u)) | (((lane >> 3) & ((1u << (bits - low)) - 1u)) << low);
        const uint32_t row0 = ((lane >> low) & ((1u << mid) - 1u)) | ((lane >> (3u + bits - low)) << mid);
        constexpr uint32_t rows_a_load = 32 / S::pieces;
        // Pages of this warp's keys of the step to load, as the table has them.
        uint32_t page[2] = {0, 0};
        auto pages = [&]() {
            const uint32_t key = (step << S::log) + dw * S::mine;
            page[0] = key < w.keys ? table_entry(a.c, w.b, key) : a.c.pages;
            page[1] = S::mine > 16 && a.c.page_log == 4u && key + 16u < w.keys ? table_entry(a.c, w.b, key + 16u) : a.c.pages;
        };
        // MXFP8: a key's scales.
        auto read_scales = [&](auto &s, const uint8_t *p, bool in) {
            if (S::blocks == 2)
                s[0] = in ? __ldg(reinterpret_cast<const uint16_t *>(p)) : 0u;
            else if (S::blocks == 4)
                s[0] = in ? __ldg(reinterpret_cast<const uint32_t *>(p)) : 0u;
            else {
                const uint2 x = in ? __ldg(reinterpret_cast<const uint2 *>(p)) : make_uint2(0u, 0u);
                s[0] = x.x;
                s[sizeof(s) / 4 - 1] = x.y;
            }
        };
        auto key_scales = [&](uint64_t at, bool in) {
            if constexpr (!S::fp4) {
                read_scales(raw.s, scales + at * S::blocks, in);
                if (S::subs == 2 && !values)
                    read_scales(raw.v, a.c.v_scales + at * S::blocks, in);
            }
        };
        auto load = [&]() {
            const uint32_t key = (step << S::log) + dw * S::mine, mask = (1u << a.c.page_log) - 1u;
            if (key + S::mine <= w.keys && page[0] < a.c.pages && (S::mine <= 16 || a.c.page_log > 4u)) {
                // all of them, one behind the other
                const uint64_t at = (((uint64_t)page[0] * a.c.heads + w.head) << a.c.page_log) + (key & mask) + row0;
                const uint8_t *c = codes + at * S::row + piece0 * 16u, *sc = scales + at * S::blocks;
#pragma unroll
                for (uint32_t i = 0; i < S::loads; ++i)
                    raw.c[i] = __ldg(reinterpret_cast<const uint4 *>(c + i * 512u));
                if constexpr (S::fp4) {
#pragma unroll
                    for (uint32_t i = 0; i < S::loads; ++i)
                        raw.s[i] = __ldg(reinterpret_cast<const uint16_t *>(sc + i * rows_a_load * S::blocks) + piece0);
                } else
                    key_scales(at - row0 + lane % S::mine, true);
                return;
            }
            const bool short_pages = S::mine > 16 && a.c.page_log == 4u;
            if ((key < w.keys && page[0] >= a.c.pages) || (short_pages && key + 16u < w.keys && page[1] >= a.c.pages))
                atomicOr(a.c.status, MXQ_DEV_INVALID_PAGE);
#pragma unroll
            for (uint32_t i = 0; i < S::loads; ++i) {
                const uint32_t row = row0 + i * rows_a_load, pg = short_pages && row >= 16u ? page[1] : page[0];
                const bool in = key + row < w.keys && pg < a.c.pages;
                const uint64_t at = in ? (((uint64_t)pg * a.c.heads + w.head) << a.c.page_log) + ((key + row) & mask) : 0ull;
                raw.c[i] = in ? __ldg(reinterpret_cast<const uint4 *>(codes + at * S::row) + piece0) : make_uint4(0u, 0u, 0u, 0u);
                if constexpr (S::fp4)
                    raw.s[i] = in ? __ldg(reinterpret_cast<const uint16_t *>(scales + at * S::blocks) + piece0) : 0u;
            }
            if constexpr (!S::fp4) {
                const uint32_t row = lane % S::mine, pg = short_pages && row >= 16u ? page[1] : page[0];
                const bool in = key + row < w.keys && pg < a.c.pages;
                const uint64_t at = in ? (((uint64_t)pg * a.c.heads + w.head) << a.c.page_log) + ((key + row) & mask) : 0ull;
                key_scales(at, in);
            }
        };
        // The chunk into its f16 tile.  top: see attention_rows.cu.
        auto store = [&](uint32_t top, uint32_t chunk, char *tile) {
            char *line0 = tile + (piece0 >> low) * S::panel + (chunk * S::mine + row0) * 128u;
#pragma unroll
            for (uint32_t i = 0; i < S::loads; ++i) {
                const uint32_t cw[4] = {raw.c[i].x, raw.c[i].y, raw.c[i].z, raw.c[i].w};
                const uint32_t turn = (row0 + i * rows_a_load) & 7u, at = (piece0 & ((1u << low) - 1u)) * (8u >> low);
                char *line = line0 + i * rows_a_load * 128u;
                if (S::fp4) {
                    const uint32_t sc = e4m3x2_to_f16x2(raw.s[i]);
                    const uint32_t sc0 = __byte_perm(sc, 0, 0x1010), sc1 = __byte_perm(sc, 0, 0x3232);
#pragma unroll
                    for (uint32_t j = 0; j < 4; ++j) {
                        uint32_t h[4];
                        e2m1x8_unpack(cw[j], h);
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            h[u] = hmul2_bits(h[u], j < 2 ? sc0 : sc1);
                        *reinterpret_cast<uint4 *>(line + (((at + j) ^ turn) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                } else {
                    uint32_t b = __shfl_sync(0xFFFFFFFFu, raw.s[0], row0 + i * rows_a_load);
                    if (S::blocks == 8) {
                        const uint32_t hi = __shfl_sync(0xFFFFFFFFu, raw.s[sizeof(raw.s) / 4 - 1], row0 + i * rows_a_load);
                        b = piece0 & 8u ? hi : b;
                    }
                    b = (b >> ((piece0 & 6u) * 4u)) & 0xFFu;       // of 32 values: two pieces
                    const float f = __uint_as_float((uint32_t)max((int)(b + 134u) - (int)top, 0) << 23);
                    const uint32_t sc = half2_bits(f, f);
#pragma unroll
                    for (uint32_t j = 0; j < 2; ++j) {
                        uint32_t h[4];
                        e4m3x4_unpack(cw[2 * j], h[0], h[1]);
                        e4m3x4_unpack(cw[2 * j + 1], h[2], h[3]);
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            h[u] = hmul2_bits(h[u], sc);
                        *reinterpret_cast<uint4 *>(line + (((at + j) ^ turn) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                }
            }
        };
        if (more) {
            pages();
            load();
        }
        while (more) {
            uint32_t top = 0, vtop = 0;     // what the chunk's codes are relative to; of the values
            if (!S::fp4 && !values) {
                uint32_t m = raw.s[0];
#pragma unroll
                for (uint32_t i = 1; i < sizeof(raw.s) / 4; ++i)
                    m = __vmaxu4(m, raw.s[i]);
                top = largest(m);
                if (S::subs == 2)
                    vtop = largest(raw.v[0]);
            }
            if (!S::fp4 && values) {
                bool ok = true;
#pragma unroll
                for (uint32_t n = 0; n < kPass; ++n)
                    if (passed[n].on && ok) {
                        ok = wait_all(&bars.tfull[passed[n].t % kRing], passed[n].t / kRing, bars, a);
                        uint32_t m = bars.vtop[passed[n].t % kRing];
                        if (S::subs == 1) {     // (warps of keys are not far enough ahead to need it)
                            __syncwarp();
                            if (lane == 0)
                                mbar_arrive(&bars.tempty[passed[n].t % kRing]);
                        }
                        m = __vmaxu4(m, m >> 16);
                        if (passed[n].first)
                            vref = ValueRef();
                        vref.follow(max(m & 0xFFu, (m >> 8) & 0xFFu), 4u);
                    }
                if (!ok)
                    break;
                top = vref.ref;
            }
            // The next chunk's place; its pages are on the way while this one is stored.
            const uint32_t now = t, chunk = dw;
            dw += stride;
            settle();
            if (more)
                pages();
            // a fresh barrier passes the wait for its odd phase
            if (!wait_all(&empty[now % S::stages], now / S::stages + 1u, bars, a))
                break;
            if (!S::fp4 && lane == 0) {         // the slots were read long ago (kRing)
                if (values)
                    bars.vref[now % kRing] = top;       // of every chunk the same
                else {
                    bars.kfac[now % kRing][chunk] = __uint_as_float(top << 23) * 0x1p-7f;
                    if (S::subs == 2) {
                        reinterpret_cast<uint8_t *>(&bars.vtop[now % kRing])[chunk] = (uint8_t)vtop;
                        mbar_arrive(&bars.tfull[now % kRing]);
                    }
                }
                mbar_arrive(&bars.ffull[now % kRing]);
            }
            store(top, chunk, tiles + now % S::stages * S::tile);
            fence_proxy_async_smem();
            __syncwarp();
            const bool held = a.stall == 1u + 2u * now + values && blockIdx.x == 0 && chunk == 0;
            if (lane == 0 && !held)
                mbar_arrive(&full[now % S::stages]);
            if (more)
                load();
        }
    } else {                                         // softmax: a row a thread
        const uint32_t wg = warp >> 2, r = (warp & 3u) * 32u + lane, lanes = ((warp & 3u) * 32u) << 16;
        char *qs = smem + wg * S::qbytes;
        uint32_t t0 = 0, buf0[kBufs] = {0, 0, 0, 0}, pv0 = 0, pieces = 0, met = 0;
        bool ok = wg < S::subs;
        // Both groups, before and after a piece that one of them has to itself: a wait for
        // a barrier's phase is one only for those who have seen the phase before it.
        auto meet = [&]() {
            if (S::subs == 2 && ok) {
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bars.meet);
                ok = wait_all(&bars.meet, met++, bars, a, kIdle);
            }
        };
        for (bool more = W::begin(w, sa, range); more && ok; more = W::next(w, sa)) {
            const Units<S> un(w);
            if (!un.two)
                meet();
            if (!ok)
                break;
            if (wg == 0 || un.two) {
                // The query's row in f16 times its factor; the sign of the scale goes with it.
                const uint32_t row = w.rt * S::rows + wg * 128u + r;
                const uint32_t i = fastdiv(row, a.groupdiv), h = w.head * a.group + row - i * a.group;
                const bool in = row < w.s.rows;
                const uint4 *src = reinterpret_cast<const uint4 *>(a.q + (int64_t)(w.s.first + (in ? i : 0u)) * a.q_stride +
                                                                   (uint64_t)(in ? h : 0u) * D);
                uint32_t m = 0;
#pragma unroll 8
                for (uint32_t k = 0; k < D / 8; ++k) {
                    const uint4 v = __ldg(src + k);
                    m = absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(m, v.x), v.y), v.z), v.w);
                }
                float f = row_factor(fold_halves(m) << 16);
                float fq = fabsf(a.scale) / f;
                if (S::fp4)
                    fq = fmaxf(fq * __ldg(a.c.k_s2 + w.head), 0x1p-126f);
                f = a.scale < 0.0f ? -f : f;
#pragma unroll 4
                for (uint32_t k = 0; k < D / 8; ++k) {
                    const uint4 v = __ldg(src + k);
                    *reinterpret_cast<uint4 *>(qs + (k >> 3) * S::qpanel + r * 128u + (((k & 7u) ^ (r & 7u)) << 4)) =
                        make_uint4(half2_bits(bf16_lo(v.x) * f, bf16_hi(v.x) * f), half2_bits(bf16_lo(v.y) * f, bf16_hi(v.y) * f),
                                   half2_bits(bf16_lo(v.z) * f, bf16_hi(v.z) * f), half2_bits(bf16_lo(v.w) * f, bf16_hi(v.w) * f));
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bars.qfull[wg]);

                // The last key of the piece that the row sees; rows past the sequence's see
                // every one, and are not stored.
                const int64_t base = (int64_t)w.k0 << S::log, pos = in ? w.s.len - w.s.n + i : 0x7FFFFFFFll;
                const int last = (int)max(min(pos, (int64_t)w.keys - 1) - base, (int64_t)-1);
                float mx = kLowest, sum = 0.0f;
                ValueRef vref;
                const uint32_t steps = un.steps;
                const bool two = un.two;
                // phases of this group's buffers: of the even ones and the odd ones of its units
                const uint32_t p0 = two ? (wg ? buf0[1] : buf0[0]) : 0u, p1 = two ? (wg ? buf0[3] : buf0[2]) : 0u;
                for (uint32_t j = 0; j < steps; ++j) {
                    const uint32_t u = two ? 2u * j + wg : j, buf = u % kBufs, t = t0 + j;
                    const uint32_t phase = two ? (j & 1u ? p1 : p0) + (j >> 1)
                                               : (buf & 2u ? (buf & 1u ? buf0[3] : buf0[2]) : (buf & 1u ? buf0[1] : buf0[0])) + (j >> 2);
                    const uint32_t at = tmem + buf * S::keys + lanes;
                    ok = S::fp4 || wait_all(&bars.ffull[t % kRing], t / kRing, bars, a);
                    if (!ok)
                        break;
                    float alpha = 1.0f;     // factor of the output so far
                    if constexpr (!S::fp4)
                        alpha = vref.move(bars.vref[t % kRing]);
                    ok = wait_all(&bars.sfull[buf], phase, bars, a);
                    if (!ok)
                        break;
                    fence_after();
                    constexpr int parts = S::keys / 32;         // of 32 columns
                    constexpr int groups = S::chunks;           // of columns whose powers are the same
                    // Keys from `lim` + 1 on the row does not see.
                    const int lim = last - (int)(j << S::log);
                    const bool cut = __any_sync(0xFFFFFFFFu, lim < (int)S::keys - 1);
                    // Of a chunk's columns: powers of the keys (with the row's own factor, kept above
                    // 0, which times -Inf would be NaN).
                    auto fac = [&](int g) { return S::fp4 ? fq : fmaxf(fq * bars.kfac[t % kRing][g], 0x1p-126f); };
                    // Weights against the reference so far, unless a row's lie more than kLag above
                    // it; then (and at first) the maximum is found first, and the weights
                    // from the scores again.  (One copy of each loop: cold instruction caches are
                    // what a short call waits for.)
                    uint32_t p[groups][S::mine / 2];
                    float total, high;
#pragma unroll 1
                    for (bool find = j == 0;;) {
                        uint32_t v[parts][32];
#pragma unroll
                        for (int c = 0; c < parts; ++c)
                            tmem_ld32(at + c * 32, v[c]);
#pragma unroll
                        for (int c = 0; c < parts; ++c)
                            tmem_ld_wait(v[c]);
                        if (cut) {
#pragma unroll
                            for (int x = 0; x < (int)S::keys; ++x)
                                v[x / 32][x % 32] = x <= lim ? v[x / 32][x % 32] : 0xFF800000u;        // -Inf
                        }
                        if (find) {
                            float top = -INFINITY;
#pragma unroll
                            for (int g = 0; g < groups; ++g) {
                                float m = -INFINITY;
#pragma unroll
                                for (int x = 0; x < (int)S::mine; ++x) {
                                    const int col = g * S::mine + x;
                                    m = fmaxf(m, __uint_as_float(v[col / 32][col % 32]));
                                }
                                top = fmaxf(top, __fmul_rn(m, fac(g)));
                            }
                            if (top - mx > kLag) {      // the weights' own difference, rounded as theirs
                                top -= kTop;
                                const float f = ex2(mx - top);
                                mx = top;
                                sum *= f;
                                alpha *= f;
                            }
                        }
                        total = 0.0f;
                        high = -INFINITY;
#pragma unroll
                        for (int g = 0; g < groups; ++g) {
                            const float fg = fac(g);
                            const float2 f2 = make_float2(fg, fg);
                            float2 part = make_float2(0.0f, 0.0f);
#pragma unroll
                            for (int x = 0; x < (int)S::mine / 2; ++x) {
                                const int col = g * S::mine + 2 * x;
                                float2 s = make_float2(__uint_as_float(v[col / 32][col % 32]), __uint_as_float(v[col / 32][col % 32 + 1]));
                                // Rounded as the maximum was, so that no weight is above 2^kLag whatever the
                                // scores' size (in one operation, 4 % faster with MXFP8, scores past 2^28
                                // could give weights without bound).  A packed product and sum are made one
                                // operation by the compiler; with a zero added there is nothing to join.
                                s = __fadd2_rn(__ffma2_rn(s, f2, make_float2(0.0f, 0.0f)), make_float2(-mx, -mx));
                                high = fmaxf(fmaxf(high, s.x), s.y);
                                s.x = ex2(s.x);
                                s.y = ex2(s.y);
                                part = __fadd2_rn(part, s);
                                p[g][x] = half2_bits(s.x, s.y);
                            }
                            total += part.x + part.y;
                        }
                        if (find || !__any_sync(0xFFFFFFFFu, high > kLag))
                            break;
                        find = true;
                    }
                    sum += total;
#pragma unroll
                    for (int g = 0; g < groups; ++g) {
                        if constexpr (S::mine == 32)
                            tmem_st16(at + g * 16, p[g]);
                        else
                            asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                                         ::"r"(at + g * 8), "r"(p[g][0]), "r"(p[g][1]), "r"(p[g][2]), "r"(p[g][3]),
                                           "r"(p[g][4]), "r"(p[g][5]), "r"(p[g][6]), "r"(p[g][7]) : "memory");
                    }
                    // Where a reference has moved the output is rescaled, once the product before
                    // this one is done.  (A wait is for a barrier's next phase.  Of two groups each has
                    // two buffers of scores, so with these scores the product before that one is done;
                    // a group alone has four, and waits at every step.)
                    const bool moved = j > 0 && __any_sync(0xFFFFFFFFu, alpha != 1.0f);
                    if (j > 0 && (moved || !two)) {
                        if (!(ok = wait_all(&bars.pv[wg], pv0 + j - 1u, bars, a)))
                            break;
                    }
                    if (moved) {
                        fence_after();
                        const uint32_t out = tmem + kOut + wg * D + lanes;
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(out + c * 32, o);
                            tmem_ld_wait(o);
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
                            tmem_st32(out + c * 32, o);
                        }
                    }
                    tmem_st_wait();
                    fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&bars.pfull[buf]);
                }
                if (!ok)
                    break;
                // The tile's output, or this CTA's part of it.
                if (!(ok = wait_all(&bars.odone[wg], pieces++, bars, a)))
                    break;
                fence_after();
                const uint32_t out = tmem + kOut + wg * D + lanes, row1 = w.rt * S::rows + wg * 128u + r;
                const uint32_t i1 = fastdiv(row1, a.groupdiv), h1 = w.head * a.group + row1 - i1 * a.group;
                const bool in1 = row1 < w.s.rows, whole = w.whole();
                const uint64_t to = (uint64_t)(w.s.first + i1) * (a.c.heads * a.group) + h1;
                float *part = part_of<S::rows, D>(a, blockIdx.x, w.slot());
                // A part is its own keys' output (the join has the factor of NVFP4); with those of the
                // pieces before, of the same tile, which this thread has left.
                float4 *rowp = reinterpret_cast<float4 *>(part + (wg * 128u + r) * D);
                float2 *statp = reinterpret_cast<float2 *>(part + S::rows * D + (wg * 128u + r) * 2u);
                float f2 = inverse(sum), unit = S::fp4 ? 1.0f : vref.unit();
                if (w.earlier()) {
                    const float2 st = add_earlier<D>(out, rowp, statp, mx, sum, unit);
                    mx = st.x;
                    sum = st.y;
                    f2 = unit = 1.0f;
                }
                if (S::fp4 && whole)
                    f2 *= __ldg(a.c.v_s2 + w.head);
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32(out + c * 32, o);
                    tmem_ld_wait(o);
                    if (in1) {
                        if (whole) {
                            uint4 *dst = reinterpret_cast<uint4 *>(a.o + to * D + c * 32);
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                uint32_t b[4];
#pragma unroll
                                for (int y = 0; y < 4; ++y) {
                                    const __nv_bfloat162 p = __floats2bfloat162_rn(__uint_as_float(o[x * 8 + y * 2]) * f2 * unit,
                                                                                  __uint_as_float(o[x * 8 + y * 2 + 1]) * f2 * unit);
                                    b[y] = *reinterpret_cast<const uint32_t *>(&p);
                                }
                                dst[x] = make_uint4(b[0], b[1], b[2], b[3]);
                            }
                        } else {
#pragma unroll
                            for (int x = 0; x < 8; ++x)
                                rowp[c * 8 + x] = make_float4(__uint_as_float(o[x * 4]) * f2 * unit, __uint_as_float(o[x * 4 + 1]) * f2 * unit,
                                                              __uint_as_float(o[x * 4 + 2]) * f2 * unit, __uint_as_float(o[x * 4 + 3]) * f2 * unit);
                        }
                    }
                    __syncwarp();       // (the next read is the whole warp's)
                }
                if (in1 && whole && a.lse)
                    a.lse[to] = sum == 0.0f ? -INFINITY : (mx + log2f(sum)) * kLn2;
                if (in1 && !whole)
                    *statp = make_float2(mx, sum);
                fence_before();     // the loads of the output, before the next tile's products
            }
            if (threadIdx.x == 0 && w.unfinished()) {
                Unfinished u = {};
                u.first = w.s.first;
                u.row0 = w.rt * S::rows;
                u.rows = w.s.rows;
                u.head = w.head;
                u.parts = parts_of(range, w.steps, w.k1);
                a.left[blockIdx.x] = u;
            }
            t0 += un.steps;
#pragma unroll
            for (uint32_t i = 0; i < kBufs; ++i)
                buf0[i] += un.uses(i);
            pv0 += un.products(wg);
            if (!un.two)
                meet();
        }
    }
    // Whichever way a warp came here, what it stored into TMEM is there before TMEM is given back.
    __syncwarp();
    tmem_st_wait();
    fence_before();
    __syncthreads();
    if (warp == 0) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512));
    }
}

namespace {

template <int FMT, int D>
cudaError_t run(AttArgs a, uint32_t ctas, cudaStream_t s)
{
    using S = Shape<FMT, D>;
    a.stall = g_stall_attention.load() ? (uint32_t)g_stall_attention.exchange(0) : 0u;
    a.spin = a.stall ? kStalledSpin : kSpin;
    const auto k = attention_tiles_kernel<FMT, D>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::smem);
    return e != cudaSuccess ? e : launch_dependent(k, dim3(ctas), kThreads, S::smem, s, a);
}

} // namespace

cudaError_t launch_attention_tiles(const AttArgs &a, int fmt, int dim, uint32_t ctas, cudaStream_t s)
{
    if (fmt == MXQ_FMT_NVFP4)
        return dim == 64    ? run<MXQ_FMT_NVFP4, 64>(a, ctas, s)
               : dim == 128 ? run<MXQ_FMT_NVFP4, 128>(a, ctas, s)
                            : run<MXQ_FMT_NVFP4, 256>(a, ctas, s);
    return dim == 64    ? run<MXQ_FMT_MXFP8, 64>(a, ctas, s)
           : dim == 128 ? run<MXQ_FMT_MXFP8, 128>(a, ctas, s)
                        : run<MXQ_FMT_MXFP8, 256>(a, ctas, s);
}

} // namespace mxq

extern "C" MXQ_API void mxq_test_stall_next_attention(int on)
{
    mxq::g_stall_attention.store(on > 0 ? on : 0);
}
