// attention_tiles.cu -- attention over a quantized cache where a sequence has many
// rows: chunks of a prompt (sm_100a).  The products are the work.
//
// A tile is 256 rows (128 for heads of 256 values) of one sequence and key/value
// head, a step 128 keys (64); attention.cuh divides them among one CTA an SM.  Both
// products run on tcgen05: S = Q K^T from shared memory into TMEM, O += P V with P
// from TMEM.  Four warps decode the cache's codes straight from global memory into
// f16 tiles in shared memory (two stages of keys, two of values, the same layout for
// both: rows of a token, 128 bytes wide, 128-byte swizzle; the values' is read as an
// MN-major operand, so nothing is transposed).  Two groups of four warps take the
// softmax of 128 rows each, a row a thread, so a row's maximum and sum need no
// exchange; while one works the tensor cores do the other's products.  One warp
// issues.  A step of 128 x 128 products costs the tensor cores 512 cycles twice, and
// a group 128 x 128 exponentials, at 16 a cycle 1024 cycles: both are near full.
//
// A unit u is a softmax and its two products.  With two groups at work unit u is
// step u / 2 of group u % 2, with one (tiles of up to 128 rows) step u; either way its
// scores are in TMEM buffer u % 2, and S of unit u + 2 is issued behind P V of unit u,
// which has read the weights that lie over the scores.
//
// The output in TMEM is rescaled only where the maximum has grown by more than 2^8
// (by the softmax group, which has the output to itself between its products);
// weights are at most 2^8 then, exact powers of two apart from what they would be.
// MXFP8 powers: as in attention_rows.cu, a largest one for every 32 (16) keys.
//
// Every wait is bounded (MXQ_DEV_WAIT_TIMEOUT); all roles then leave, the issuing
// one behind its last product.
#include "attention.cuh"
#include "mxq_mma.cuh"
#include "mxq_tcgen05.cuh"
#include <algorithm>

namespace mxq {

namespace {

constexpr uint32_t kSpin = 1u << 18;        // tests of a barrier before a wait gives up
// Warps 0-3 and 4-7: softmax groups, whose first warps issue; 8-11 decode keys,
// 12-15 values.
constexpr uint32_t kCodeWarp = 8;
constexpr int kThreads = 512;
// Registers of a thread: 128 at launch, of which the decoding warps give up what the
// softmax ones take.
constexpr int kLaunchRegs = 128, kSoftRegs = 192, kCodeRegs = 64;
static_assert(kLaunchRegs * kThreads <= 65536 && kSoftRegs + kCodeRegs <= 2 * kLaunchRegs, "register shares");

template <int FMT, int D>
struct Shape {
    static constexpr bool fp4 = FMT == MXQ_FMT_NVFP4;
    static constexpr uint32_t row = fp4 ? D / 2 : D;            // bytes of a token's codes
    static constexpr uint32_t blocks = fp4 ? D / 16 : D / 32;   // and of its scales
    static constexpr uint32_t log = D == 256 ? 6 : 7, keys = 1u << log;
    static constexpr uint32_t mine = keys / 4;                  // keys of a decoding warp
    static constexpr uint32_t subs = D == 256 ? 1 : 2, rows = 128 * subs;
    static constexpr uint32_t panel = keys * 128;               // 64 values of a step's tokens
    static constexpr uint32_t qpanel = 128 * 128;
    static constexpr uint32_t qbytes = 128 * D * 2, tile = keys * D * 2;
    static constexpr uint32_t smem = subs * qbytes + 4 * tile + 1024;
    static constexpr uint32_t pieces = row / 16;                // of a token's codes
    static constexpr uint32_t loads = mine * pieces / 32;       // pieces of a lane
};

struct Bars {
    uint64_t kfull[2], kempty[2], vfull[2], vempty[2], sfull[2], pfull[2], pv[2], qfull[2], ffull[4], meet, drain[2];
    uint32_t tmem, abort;
    float kfac[4][4], vexp[4][4], vinv[4][4];   // by step % 4 and decoding warp: powers of keys, values
};

__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, Bars &s, uint32_t *status)
{
    for (uint32_t i = 0; i < kSpin; ++i) {
        if (mbar_try_wait(bar, parity & 1u))
            return true;
        if ((i & 63u) == 63u && *reinterpret_cast<volatile uint32_t *>(&s.abort))
            return false;
    }
    *reinterpret_cast<volatile uint32_t *>(&s.abort) = 1u;
    atomicOr(status, MXQ_DEV_WAIT_TIMEOUT);
    return false;
}
// The whole warp.
__device__ __forceinline__ bool wait_all(uint64_t *bar, uint32_t parity, Bars &s, uint32_t *status)
{
    return __all_sync(0xFFFFFFFFu, wait_bar(bar, parity, s, status));
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

// How the units of a piece lie: `two` groups, or the first alone.
template <typename S>
struct Units {
    bool two;
    uint32_t steps;
    template <typename W>
    __device__ __forceinline__ Units(const W &w)
        : two(S::subs == 2 && min(w.s.rows - w.rt * S::rows, S::rows) > 128u), steps(w.k1 - w.k0) {}
    // Uses of TMEM buffer i.
    __device__ __forceinline__ uint32_t uses(uint32_t i) const { return two ? steps : (steps + 1u - i) >> 1; }
    // Products with the values of group i.
    __device__ __forceinline__ uint32_t products(uint32_t i) const { return two || i == 0 ? steps : 0u; }
};

// A decoding warp's part of a step: pieces of codes and their scales, in registers.
template <int FMT, int D>
struct Raw {
    uint4 c[Shape<FMT, D>::loads];
    uint32_t s[Shape<FMT, D>::loads];       // MXFP8: a byte; NVFP4: two
};

} // namespace

template <int FMT, int D>
__global__ void __launch_bounds__(kThreads, 1)
attention_tiles_kernel(const AttArgs a)
{
    using S = Shape<FMT, D>;
    using W = Walk<S::rows, S::log>;
    extern __shared__ __align__(1024) char smem_raw[];
    __shared__ Bars bars;
    __shared__ Range range;
    char *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    char *kt = smem + S::subs * S::qbytes, *vt = kt + 2 * S::tile;
    const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31u;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.kfull[i], 4);
            mbar_init(&bars.kempty[i], 2);
            mbar_init(&bars.vfull[i], 4);
            mbar_init(&bars.vempty[i], 2);
            mbar_init(&bars.sfull[i], 1);
            mbar_init(&bars.pfull[i], 4);
            mbar_init(&bars.pv[i], 1);
            mbar_init(&bars.qfull[i], 4);
            mbar_init(&bars.drain[i], 1);
        }
        for (int i = 0; i < 4; ++i)
            mbar_init(&bars.ffull[i], 8);
        mbar_init(&bars.meet, 8);
        bars.abort = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_addr(&bars.tmem)), "n"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();
    find_range<typename W::Div>(a, range);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = bars.tmem;
    if (threadIdx.x == 0)
        a.left[blockIdx.x].parts = 0u;
    // TMEM columns: scores in two buffers, outputs, weights.  With heads of 128 values
    // there is no room for the weights but over the scores that they come from.
    constexpr uint32_t kOut = 2 * S::keys;
    constexpr uint32_t kP = D == 128 ? 0 : kOut + S::subs * D, kPStride = D == 128 ? S::keys : S::keys / 2;
    static_assert(D == 128 || kP + S::keys <= 512, "TMEM");

    W w;
    if (warp >= kCodeWarp) {                         // decoding
        regs_down<kCodeRegs>();
        const bool values = warp >= kCodeWarp + 4u;
        const uint32_t dw = warp & 3u;
        const uint8_t *codes = values ? a.c.v_codes : a.c.k_codes, *scales = values ? a.c.v_scales : a.c.k_scales;
        uint64_t *full = values ? bars.vfull : bars.kfull, *empty = values ? bars.vempty : bars.kempty;
        char *tiles = values ? vt : kt;
        Raw<FMT, D> raw;
        bool more = w.begin(a, range);
        uint32_t step = w.k0;
        const uint32_t row0 = lane / S::pieces, piece0 = lane % S::pieces;      // of the lane's first load
        constexpr uint32_t rows_a_load = 32 / S::pieces;
        // Pages of this warp's keys of the step to load; c.pages: none.
        uint32_t page[2] = {0, 0};
        auto pages = [&]() {
            const uint32_t key = (step << S::log) + dw * S::mine;
            page[0] = key < w.keys ? find_page(a.c, w.b, key) : a.c.pages;
            page[1] = page[0];
            if (S::mine > 16 && a.c.page_log == 4u)
                page[1] = key + 16u < w.keys ? find_page(a.c, w.b, key + 16u) : a.c.pages;
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
#pragma unroll
                for (uint32_t i = 0; i < S::loads; ++i)
                    raw.s[i] = S::fp4 ? __ldg(reinterpret_cast<const uint16_t *>(sc + i * rows_a_load * S::blocks) + piece0)
                                      : __ldg(sc + i * rows_a_load * S::blocks + (piece0 >> 1));
                return;
            }
#pragma unroll
            for (uint32_t i = 0; i < S::loads; ++i) {
                const uint32_t row = row0 + i * rows_a_load, pg = page[S::mine > 16 ? row >> 4 : 0];
                const bool in = key + row < w.keys && pg < a.c.pages;
                const uint64_t at = in ? (((uint64_t)pg * a.c.heads + w.head) << a.c.page_log) + ((key + row) & mask) : 0ull;
                raw.c[i] = in ? __ldg(reinterpret_cast<const uint4 *>(codes + at * S::row) + piece0) : make_uint4(0u, 0u, 0u, 0u);
                raw.s[i] = !in      ? 0u
                           : S::fp4 ? __ldg(reinterpret_cast<const uint16_t *>(scales + at * S::blocks) + piece0)
                                    : __ldg(scales + at * S::blocks + (piece0 >> 1));
            }
        };
        // One tensor's part of a step into its f16 tile.  top: see attention_rows.cu.
        auto store = [&](uint32_t top, char *tile) {
#pragma unroll
            for (uint32_t i = 0; i < S::loads; ++i) {
                const uint32_t row = dw * S::mine + row0 + i * rows_a_load, piece = piece0;
                const uint32_t cw[4] = {raw.c[i].x, raw.c[i].y, raw.c[i].z, raw.c[i].w};
                if (S::fp4) {
                    uint32_t sc0 = e4m3x2_to_f16x2(raw.s[i]), sc1 = __byte_perm(sc0, 0, 0x3232);
                    sc0 = __byte_perm(sc0, 0, 0x1010);
                    uint32_t h[4][4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        e2m1x8_unpack(cw[j], h[j]);
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            h[j][u] = hmul2_bits(h[j][u], j < 2 ? sc0 : sc1);
                    }
                    char *line = tile + (piece >> 1) * S::panel + row * 128u;
                    // 4 pieces of 16 bytes; lanes whose pieces would meet on a bank take them in another order
                    const uint32_t turn = D == 64 ? 0u : piece & 2u;
#pragma unroll
                    for (uint32_t j = 0; j < 4; ++j) {
                        const uint32_t at = ((piece & 1u) * 4u + (j ^ turn)) ^ (row & 7u);
                        uint4 v = make_uint4(h[j][0], h[j][1], h[j][2], h[j][3]);
                        if (D != 64) {
                            const uint32_t o = j ^ 2u;
                            if (turn)
                                v = make_uint4(h[o][0], h[o][1], h[o][2], h[o][3]);
                        }
                        *reinterpret_cast<uint4 *>(line + at * 16u) = v;
                    }
                } else {
                    const float f = __uint_as_float((uint32_t)max((int)(raw.s[i] + 134u) - (int)top, 0) << 23);
                    const uint32_t sc = half2_bits(f, f);
                    uint32_t h[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        e4m3x4_unpack(cw[j], h[2 * j], h[2 * j + 1]);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        h[j] = hmul2_bits(h[j], sc);
                    char *line = tile + (piece >> 2) * S::panel + row * 128u;
                    const bool turn = D != 64 && (piece & 4u);
                    const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
                    const uint32_t at = (piece & 3u) * 2u;
                    *reinterpret_cast<uint4 *>(line + (((at + turn) ^ (row & 7u)) << 4)) = turn ? hi : lo;
                    *reinterpret_cast<uint4 *>(line + (((at + !turn) ^ (row & 7u)) << 4)) = turn ? lo : hi;
                }
            }
        };
        if (more) {
            pages();
            load();
        }
        for (uint32_t t = 0; more; ++t) {
            uint32_t top = 27u;     // 2^-100 at least: values below count as zeros
            if (!S::fp4) {
#pragma unroll
                for (uint32_t i = 0; i < S::loads; ++i)
                    top = max(top, raw.s[i]);
                top = __reduce_max_sync(0xFFFFFFFFu, top);
            }
            // The powers: a slot was read four steps ago, which a product with the values of
            // the step after that says (waited for below), and scores two steps on.
            if (!S::fp4 && values && lane == 0) {
                bars.vexp[t & 3u][dw] = (float)((int)top - 134);
                bars.vinv[t & 3u][dw] = __uint_as_float((uint32_t)(261 - (int)top) << 23);
                mbar_arrive(&bars.ffull[t & 3u]);
            }
            // the step after this one
            if (++step == w.k1) {
                more = w.next();
                step = w.k0;
            }
            if (more)
                pages();
            // a fresh barrier passes the wait for its odd phase
            if (!wait_all(&empty[t & 1u], (t >> 1) + 1u, bars, a.c.status))
                break;
            if (!S::fp4 && !values && lane == 0) {
                bars.kfac[t & 3u][dw] = __uint_as_float(top << 23) * 0x1p-7f;
                mbar_arrive(&bars.ffull[t & 3u]);
            }
            store(top, tiles + (t & 1u) * S::tile);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&full[t & 1u]);
            if (more)
                load();
        }
    } else {                                         // softmax: a row a thread
        regs_up<kSoftRegs>();
        const uint32_t wg = warp >> 2, r = (warp & 3u) * 32u + lane, lanes = ((warp & 3u) * 32u) << 16;
        char *qs = smem + wg * S::qbytes;
        const bool issuer = (warp & 3u) == 0u;
        const uint32_t one = elect_one();
        constexpr uint32_t sdesc = (1u << 4) | ((S::keys / 8u) << 17) | (8u << 24);
        constexpr uint32_t odesc = (1u << 4) | (1u << 16) | ((D / 8u) << 17) | (8u << 24);
        uint32_t t0 = 0, buf0[2] = {0, 0}, pv0 = 0, met = 0, pieces = 0;
        bool ok = wg < S::subs;
        // Both groups, before and after a piece that one of them has to itself: a wait for
        // a barrier's phase is one only for those who have seen the phase before it.
        auto meet = [&]() {
            if (S::subs == 2 && ok) {
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bars.meet);
                ok = wait_all(&bars.meet, met++, bars, a.c.status);
            }
        };
        // The issuing warp: scores of step j of the piece; then weights times values.
        // A group alone makes up for the other's arrivals.
        auto scores = [&](uint32_t j, uint32_t buf, bool two) {
            const uint32_t t = t0 + j;
            if (!(ok = ok && wait_all(&bars.kfull[t & 1u], t >> 1, bars, a.c.status)))
                return;
            fence_after();
            const uint64_t qd = operand_desc(smem_addr(qs)), kd = operand_desc(smem_addr(kt + (t & 1u) * S::tile));
#pragma unroll
            for (uint32_t k = 0; k < D / 16; ++k)
                umma_ss(tmem + buf * S::keys, qd + (k >> 2) * (S::qpanel >> 4) + (k & 3u) * 2u,
                        kd + (k >> 2) * (S::panel >> 4) + (k & 3u) * 2u, sdesc, k > 0, one);
            umma_commit(&bars.sfull[buf], one);
            umma_commit(&bars.kempty[t & 1u], one);
            if (!two)
                umma_commit(&bars.kempty[t & 1u], one);
        };
        auto products = [&](uint32_t j, uint32_t buf, uint32_t phase, bool two) {
            const uint32_t t = t0 + j;
            ok = ok && wait_all(&bars.vfull[t & 1u], t >> 1, bars, a.c.status) &&
                 wait_all(&bars.pfull[buf], phase, bars, a.c.status);
            if (!ok)
                return;
            fence_after();
            const uint64_t vd = columns_desc(smem_addr(vt + (t & 1u) * S::tile), S::panel);
#pragma unroll
            for (uint32_t k = 0; k < S::keys / 16; ++k)
                umma_ts(tmem + kOut + wg * D, tmem + kP + buf * kPStride + k * 8u, vd + k * 128u, odesc, j > 0 || k > 0, one);
            umma_commit(&bars.pv[wg], one);
            umma_commit(&bars.vempty[t & 1u], one);
            if (!two)
                umma_commit(&bars.vempty[t & 1u], one);
        };
        for (bool more = w.begin(a, range); more && ok; more = w.next()) {
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
#pragma unroll
                for (uint32_t k = 0; k < D / 8; ++k) {
                    const uint4 v = __ldg(src + k);
                    m = absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(m, v.x), v.y), v.z), v.w);
                }
                float f = row_factor(fold_halves(m) << 16);
                float fq = fabsf(a.scale) / f;
                if (S::fp4)
                    fq *= __ldg(a.c.k_s2 + w.head);
                f = a.scale < 0.0f ? -f : f;
#pragma unroll
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
                if (issuer) {
                    ok = wait_all(&bars.qfull[wg], pieces, bars, a.c.status);
                    scores(0, un.two ? wg : 0u, un.two);
                    if (!un.two && un.steps > 1u)
                        scores(1, 1, false);
                }
                ++pieces;

                // rows past the sequence's see every key, and are not stored
                const int64_t pos = in ? w.s.len - w.s.n + i : 0x7FFFFFFFll;
                float mx = kLowest, sum = 0.0f;
                const uint32_t out = tmem + kOut + wg * D + lanes;
                for (uint32_t j = 0; j < un.steps; ++j) {
                    const uint32_t buf = un.two ? wg : j & 1u, t = t0 + j;
                    const uint32_t at = tmem + buf * S::keys + lanes, to_p = tmem + kP + buf * kPStride + lanes;
                    ok = ok && (S::fp4 || wait_all(&bars.ffull[t & 3u], t >> 2, bars, a.c.status)) &&
                         wait_all(&bars.sfull[buf], buf0[buf] + (un.two ? j : j >> 1), bars, a.c.status);
                    if (!ok)
                        break;
                    fence_after();
                    constexpr int chunks = S::keys / 32;        // of 32 columns
                    constexpr int per = 32 / S::mine < 1 ? 1 : 32 / S::mine;    // powers of a chunk: 1, or 2 of 16 columns
                    uint32_t v[chunks][32];
#pragma unroll
                    for (int c = 0; c < chunks; ++c)
                        tmem_ld32(at + c * 32, v[c]);
#pragma unroll
                    for (int c = 0; c < chunks; ++c)
                        tmem_ld_wait(v[c]);
                    float fac[4], e[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        fac[c] = S::fp4 ? fq : fq * bars.kfac[t & 3u][c];
                        e[c] = S::fp4 ? 0.0f : bars.vexp[t & 3u][c];
                    }
                    const uint32_t key = (w.k0 + j) << S::log;
                    const int lim = (int)max(min(pos, (int64_t)w.keys - 1) - (int64_t)key, (int64_t)-1);
                    const bool cut = __any_sync(0xFFFFFFFFu, lim < (int)S::keys - 1);
                    float top = -INFINITY;
                    if (cut) {
#pragma unroll
                        for (int c = 0; c < chunks; ++c)
#pragma unroll
                            for (int x = 0; x < 32; ++x) {
                                const int g = c * per + x * per / 32;
                                const float s = c * 32 + x <= lim ? fmaf(__uint_as_float(v[c][x]), fac[g], e[g]) : -INFINITY;
                                v[c][x] = __float_as_uint(s);
                                top = fmaxf(top, s);
                            }
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            fac[c] = 1.0f;
                            e[c] = 0.0f;
                        }
                    } else {
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
                            for (int x = 0; x < (int)S::mine; x += 2) {
                                const int col = g * S::mine + x;
                                m0 = fmaxf(m0, __uint_as_float(v[col / 32][col % 32]));
                                m1 = fmaxf(m1, __uint_as_float(v[col / 32][col % 32 + 1]));
                            }
                            top = fmaxf(top, fmaf(fmaxf(m0, m1), fac[g], e[g]));
                        }
                    }
                    float alpha = 1.0f;
                    if (top > mx + 8.0f) {
                        alpha = ex2(mx - top);
                        mx = top;
                        sum *= alpha;
                    }
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const float2 f2 = make_float2(fac[g], fac[g]), b2 = make_float2(e[g] - mx, e[g] - mx);
                        float2 part = make_float2(0.0f, 0.0f);
                        uint32_t p[S::mine / 2];
#pragma unroll
                        for (int x = 0; x < (int)S::mine / 2; ++x) {
                            const int col = g * S::mine + 2 * x;
                            float2 s = __ffma2_rn(make_float2(__uint_as_float(v[col / 32][col % 32]),
                                                              __uint_as_float(v[col / 32][col % 32 + 1])), f2, b2);
                            s.x = ex2(s.x);
                            s.y = ex2(s.y);
                            part = __fadd2_rn(part, s);
                            p[x] = half2_bits(s.x, s.y);
                        }
                        sum = S::fp4 ? sum + (part.x + part.y) : fmaf(part.x + part.y, bars.vinv[t & 3u][g], sum);
                        if constexpr (S::mine == 32)
                            tmem_st16(to_p + g * 16, p);
                        else
                            asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                                         ::"r"(to_p + g * 8), "r"(p[0]), "r"(p[1]), "r"(p[2]), "r"(p[3]), "r"(p[4]), "r"(p[5]),
                                           "r"(p[6]), "r"(p[7]) : "memory");
                    }
                    // The product before this one is done (every phase is waited for, since a wait
                    // is for the one that comes next): the output may be rescaled.
                    if (j > 0) {
                        if (!(ok = wait_all(&bars.pv[wg], pv0 + j - 1u, bars, a.c.status)))
                            break;
                        if (__any_sync(0xFFFFFFFFu, alpha != 1.0f)) {
                            fence_after();
#pragma unroll
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
                    }
                    tmem_st_wait();
                    fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&bars.pfull[buf]);
                    if (issuer) {
                        products(j, buf, buf0[buf] + (un.two ? j : j >> 1), un.two);
                        if (un.two && j + 1u < un.steps)
                            scores(j + 1u, buf, true);
                        if (!un.two && j + 2u < un.steps)
                            scores(j + 2u, buf, false);
                        if (!ok)
                            break;
                    }
                }
                if (!ok)
                    break;
                // The tile's output, or this CTA's part of it.
                if (!(ok = wait_all(&bars.pv[wg], pv0 + un.steps - 1u, bars, a.c.status)))
                    break;
                fence_after();
                const bool whole = w.whole();
                const uint64_t to = (uint64_t)(w.s.first + i) * (a.c.heads * a.group) + h;
                float *part = part_of<S::rows, D>(a, blockIdx.x, w.k0 == 0u);
                const float f2 = sum == 0.0f ? 0.0f : (S::fp4 ? __ldg(a.c.v_s2 + w.head) : 1.0f) / sum;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32(out + c * 32, o);
                    tmem_ld_wait(o);
                    if (!in)
                        continue;
                    if (whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(a.o + to * D + c * 32);
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            uint32_t b[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const __nv_bfloat162 p = __floats2bfloat162_rn(__uint_as_float(o[x * 8 + y * 2]) * f2,
                                                                              __uint_as_float(o[x * 8 + y * 2 + 1]) * f2);
                                b[y] = *reinterpret_cast<const uint32_t *>(&p);
                            }
                            dst[x] = make_uint4(b[0], b[1], b[2], b[3]);
                        }
                    } else {
                        uint4 *dst = reinterpret_cast<uint4 *>(part + (wg * 128u + r) * D + c * 32);
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            dst[x] = make_uint4(o[x * 4], o[x * 4 + 1], o[x * 4 + 2], o[x * 4 + 3]);
                    }
                }
                if (in && whole && a.lse)
                    a.lse[to] = sum == 0.0f ? -INFINITY : (mx + log2f(sum)) * kLn2;
                if (in && !whole)
                    *reinterpret_cast<float2 *>(part + S::rows * D + (wg * 128u + r) * 2u) = make_float2(mx, sum);
                fence_before();     // the loads of the output, before the next tile's products
            }
            if (threadIdx.x == 0 && w.k0 == 0u && !w.whole()) {
                Unfinished u = {};
                u.first = w.s.first;
                u.row0 = w.rt * S::rows;
                u.rows = w.s.rows;
                u.head = w.head;
                u.parts = parts_of(range, w.steps, w.k1);
                a.left[blockIdx.x] = u;
            }
            t0 += un.steps;
            buf0[0] += un.uses(0);
            buf0[1] += un.uses(1);
            pv0 += un.products(wg);
            if (!un.two)
                meet();
        }
        if (issuer) {
            umma_commit(&bars.drain[wg], one);       // every product of this warp is done
            for (uint32_t i = 0; i < kSpin && !mbar_try_wait(&bars.drain[wg], 0); ++i)
                ;
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (warp == 0) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512));
    }
}

namespace {

template <int FMT, int D>
cudaError_t run(const AttArgs &a, uint32_t ctas, cudaStream_t s)
{
    using S = Shape<FMT, D>;
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
