// gemm.cu -- product of block-FP8 matrices (sm_100a):
//   c[m, n] = sum over K blocks kb of sa[m, kb] sb[n / 128, kb] P,
//   P = sum of a[m, k] b[n, k] over the 128 k of block kb,
// a E4M3 [M, K] with a scale per row and 128 values (a token tile), b E4M3
// [N, K] with a scale per 128 x 128 block (weights), c bf16 or fp32.
//
// The scales are fp32, not powers of two, so the block-scaled instructions
// cannot take them: every block's P (exact products, fp32 sums) is scaled and
// added to fp32 sums in registers.
//
// gemm_tile_kernel (M above kSmallM).  One persistent CTA per SM, tiles of 128
// rows by BN columns.  A producer thread fetches the 128-byte-wide K blocks of
// a and b by TMA (128-byte swizzle; rows, columns and a last K block past the
// ends arrive as zeros), one thread issues tcgen05.mma kind::f8f6f4 (four of
// K = 32 a block) into one of NB TMEM buffers, and 16 warps move each finished
// buffer into their sums: acc += (sa sb) P.  A warp has 32 rows (its TMEM
// lanes) and BN / 4 columns, so all of a thread's sums share one row scale and
// one column scale.  A scale warp brings the 128 row scales and the column
// scales of each block into shared memory ahead of time; read by the 16 warps
// themselves, 32 lines a load, they would cost as many cycles as the product.
//
// gemm_small_kernel (few rows: decoding).  The read of b is the bound.  A
// warp multiplies 16 rows of b by up to 8 NT rows of a with mma.sync
// m16n8k32; 8 warps of a CTA split K by blocks and add their sums in a fixed
// order.  Both operands come straight from global memory: a lane's 16-byte
// pieces of a row of b and of a row of a hold the same k, and the order of k
// inside a block is free.
//
// Every wait is bounded: a wait that runs into its limit sets
// MXQ_DEV_WAIT_TIMEOUT, all roles leave their loops, copies and products in
// flight are awaited (bounded) and TMEM is freed.
#include "mxq_device.cuh"
#include "mxq_internal.h"
#include "mxq.h"
#include "mxq_tma.cuh"

namespace mxq {

namespace {

// Waits give up after this many tests; a test may suspend for a while in
// hardware, so this is well above any wait that makes progress and below a
// second or two.
constexpr uint32_t kGemmSpin = 1u << 20;
constexpr int kSmallM = 64;

template <typename T>
__device__ __forceinline__ T to_out(float v);
template <>
__device__ __forceinline__ float to_out<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 to_out<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// ------------------------------------------------------------- few rows --

// c += A B: A 16 rows x 32 k, B 32 k x 8 columns, E4M3.
__device__ __forceinline__ void mma16832(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int NT, typename Out>
__global__ void __launch_bounds__(256)
gemm_small_kernel(const uint8_t *__restrict__ a, const float *__restrict__ sa, const uint8_t *__restrict__ b,
                  const float *__restrict__ sb, uint32_t M, uint32_t N, uint32_t K, Out *__restrict__ c)
{
    __shared__ float red[8][NT * 8][17];
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3u;
    const uint32_t n0 = blockIdx.x * 16u, m0 = blockIdx.y * (8u * NT), KB = (K + 127u) / 128u;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const bool r0 = n0 + g < N, r1 = n0 + g + 8u < N;
    const uint8_t *b0 = b + (uint64_t)(n0 + g) * K, *b1 = b0 + 8ull * K;
    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
        acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
#pragma unroll 2
    for (uint32_t kb = warp; kb < KB; kb += 8u) {
        const uint32_t k0 = kb * 128u + t * 16u, k1 = k0 + 64u;
        const bool p0 = k0 < K, p1 = k1 < K;
        const uint4 x0 = r0 && p0 ? __ldg(reinterpret_cast<const uint4 *>(b0 + k0)) : zero;
        const uint4 x1 = r0 && p1 ? __ldg(reinterpret_cast<const uint4 *>(b0 + k1)) : zero;
        const uint4 y0 = r1 && p0 ? __ldg(reinterpret_cast<const uint4 *>(b1 + k0)) : zero;
        const uint4 y1 = r1 && p1 ? __ldg(reinterpret_cast<const uint4 *>(b1 + k1)) : zero;
        const float wb = __ldg(sb + (uint64_t)(n0 >> 7) * KB + kb);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const uint32_t m = m0 + i * 8u + g, mc = m0 + i * 8u + t * 2u;
            const uint8_t *ar = a + (uint64_t)m * K;
            const uint4 v0 = m < M && p0 ? __ldg(reinterpret_cast<const uint4 *>(ar + k0)) : zero;
            const uint4 v1 = m < M && p1 ? __ldg(reinterpret_cast<const uint4 *>(ar + k1)) : zero;
            const float s0 = mc < M ? __ldg(sa + (uint64_t)mc * KB + kb) * wb : 0.0f;
            const float s1 = mc + 1u < M ? __ldg(sa + (uint64_t)(mc + 1u) * KB + kb) * wb : 0.0f;
            float p[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma16832(p, x0.x, y0.x, x0.y, y0.y, v0.x, v0.y);
            mma16832(p, x0.z, y0.z, x0.w, y0.w, v0.z, v0.w);
            mma16832(p, x1.x, y1.x, x1.y, y1.y, v1.x, v1.y);
            mma16832(p, x1.z, y1.z, x1.w, y1.w, v1.z, v1.w);
            acc[i][0] = fmaf(p[0], s0, acc[i][0]);
            acc[i][1] = fmaf(p[1], s1, acc[i][1]);
            acc[i][2] = fmaf(p[2], s0, acc[i][2]);
            acc[i][3] = fmaf(p[3], s1, acc[i][3]);
        }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            red[warp][i * 8 + t * 2 + (j & 1)][g + (j >> 1) * 8] = acc[i][j];
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < NT * 128u; i += 256u) {
        const uint32_t m = i >> 4, n = i & 15u;
        float s = red[0][m][n];
#pragma unroll
        for (int w = 1; w < 8; ++w)
            s += red[w][m][n];
        if (m0 + m < M && n0 + n < N)
            c[(uint64_t)(m0 + m) * N + n0 + n] = to_out<Out>(s);
    }
}

// ------------------------------------------------------------ many rows --

constexpr int kEpiWarps = 16;
constexpr int kTileThreads = 32 * (kEpiWarps + 4);   // sums, producer, product, scales, one idle warp
constexpr int kStageOut = 2048;                      // bytes a warp stages its result through

template <int BN>
struct Tile {
    static constexpr int bytes = (128 + BN) * 128;                    // one K block of a and b
    static constexpr int stages = BN == 256 ? 4 : BN == 128 ? 5 : 7;   // 227 KB in all
    static constexpr int bufs = BN == 256 ? 2 : 4;                    // TMEM buffers of BN columns
    static constexpr int cols = BN / 4;                               // a warp's columns
};

struct TileArgs {
    const float *sa, *sb;
    void *c;
    uint32_t *status;
    uint32_t M, N, K, KB;
    uint32_t mt, nt;            // tiles in each direction
    uint32_t group;             // column tiles of a group; groups are walked one after the other
};

struct TileBars {
    uint64_t full[8], empty[8], tfull[4], tempty[4], drain;
    uint32_t tmem, abort;
};

// Tile number -> row and column tile.  Inside a group of column tiles the
// columns run fastest, so that the rows of a that the CTAs share at a time are
// few and the group's part of b stays in L2.
__device__ __forceinline__ void tile_at(const TileArgs &p, uint32_t i, uint32_t &m, uint32_t &n)
{
    const uint32_t per = p.mt * p.group, grp = i / per, in = i - grp * per;
    const uint32_t w = min(p.group, p.nt - grp * p.group);
    m = in / w;
    n = grp * p.group + (in - m * w);
}

__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, TileBars &s, uint32_t *status)
{
    for (uint32_t i = 0; i < kGemmSpin; ++i) {
        if (mbar_try_wait(bar, parity))
            return true;
        if ((i & 63u) == 63u && *reinterpret_cast<volatile uint32_t *>(&s.abort))
            return false;
    }
    *reinterpret_cast<volatile uint32_t *>(&s.abort) = 1u;
    atomicOr(status, MXQ_DEV_WAIT_TIMEOUT);
    return false;
}

// Shared-memory descriptor of a K-major operand tile, rows of 128 bytes with
// the 128-byte swizzle: groups of 8 rows are 1024 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr)
{
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void umma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add) : "memory");
}

__device__ __forceinline__ void umma_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&v)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
                 "%13, %14, %15}, [%16];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                   "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]),
                   "=r"(v[15])
                 : "r"(addr));
}

__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// One warp's 32 rows x COLS sums -> global, through 2 KB of shared memory: 64
// bytes of each row at a time, their 16-byte pieces permuted against bank
// conflicts, written out in whole rows.
template <int COLS, typename Out>
__device__ __forceinline__ void store_rows(const float2 *acc, char *buf, Out *c, uint32_t m0, uint32_t n0,
                                           const TileArgs &p, uint32_t lane)
{
    constexpr int per = 64 / sizeof(Out);       // columns a round
    constexpr int rounds = (COLS + per - 1) / per;
    constexpr int used = COLS < per ? COLS : per;
    constexpr int pieces = used * (int)sizeof(Out) / 16;
    const bool vec = (p.N * sizeof(Out)) % 16 == 0;
    const uint32_t swz = (lane >> 1) & 3u;
#pragma unroll
    for (int r = 0; r < rounds; ++r) {
        __syncwarp();
#pragma unroll
        for (int q = 0; q < pieces; ++q) {
            uint4 v;
            const float2 *s = acc + (r * used + q * (16 / (int)sizeof(Out))) / 2;
            if (sizeof(Out) == 2) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(s[i].x, s[i].y);
                    w[i] = *reinterpret_cast<const uint32_t *>(&h);
                }
                v = make_uint4(w[0], w[1], w[2], w[3]);
            } else
                v = make_uint4(__float_as_uint(s[0].x), __float_as_uint(s[0].y), __float_as_uint(s[1].x),
                               __float_as_uint(s[1].y));
            *reinterpret_cast<uint4 *>(buf + lane * 64u + (((uint32_t)q ^ swz) << 4)) = v;
        }
        __syncwarp();
        const uint32_t nr = n0 + r * used;
        if (vec) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t row = i * 8u + (lane >> 2), q = lane & 3u, n = nr + q * (16u / sizeof(Out));
                if (q < pieces && m0 + row < p.M && n < p.N)
                    *reinterpret_cast<uint4 *>(c + (uint64_t)(m0 + row) * p.N + n) =
                        *reinterpret_cast<const uint4 *>(buf + row * 64u + ((q ^ ((row >> 1) & 3u)) << 4));
            }
        } else {
            for (uint32_t i = lane; i < 32u * used; i += 32u) {
                const uint32_t row = i / used, col = i % used, q = col * (uint32_t)sizeof(Out) / 16u;
                if (m0 + row < p.M && nr + col < p.N)
                    c[(uint64_t)(m0 + row) * p.N + nr + col] = *reinterpret_cast<const Out *>(
                        buf + row * 64u + ((q ^ ((row >> 1) & 3u)) << 4) + (col * sizeof(Out)) % 16u);
            }
        }
    }
}

} // namespace

template <int BN, typename Out>
__global__ void __launch_bounds__(kTileThreads, 1)
gemm_tile_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb, const TileArgs p)
{
    using T = Tile<BN>;
    extern __shared__ __align__(1024) char smem_raw[];
    __shared__ TileBars bars;
    __shared__ float srow[T::bufs][128], scol[T::bufs][4];
    // operand tiles start on 1024-byte boundaries (the swizzle repeats there)
    char *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
    const uint32_t ntile = p.mt * p.nt;
    if (threadIdx.x == 0) {
        for (int i = 0; i < T::stages; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < T::bufs; ++i) {
            mbar_init(&bars.tfull[i], 2);            // the product and the scales
            mbar_init(&bars.tempty[i], kEpiWarps);
        }
        mbar_init(&bars.drain, 1);
        bars.abort = 0;
        fence_mbar_init();
    }
    if (warp == kEpiWarps + 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_addr(&bars.tmem)), "n"(T::bufs * BN) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = bars.tmem;

    if (warp == kEpiWarps) {                         // producer
        if (lane == 0) {
            uint32_t s = 0, ph = 1;                  // a fresh barrier passes the wait for its odd phase
            bool ok = true;
            for (uint32_t i = blockIdx.x; i < ntile && ok; i += gridDim.x) {
                uint32_t m, n;
                tile_at(p, i, m, n);
                for (uint32_t kb = 0; kb < p.KB; ++kb) {
                    if (!(ok = wait_bar(&bars.empty[s], ph, bars, p.status)))
                        break;
                    char *dst = smem + s * T::bytes;
                    mbar_arrive_expect_tx(&bars.full[s], T::bytes);
                    tma_load_2d(dst, &ma, kb * 128u, m * 128u, &bars.full[s]);
                    tma_load_2d(dst + 128 * 128, &mb, kb * 128u, n * BN, &bars.full[s]);
                    if (++s == T::stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok) {
                // copies in flight: the last fill of every stage.  Stages
                // before s were filled in the current pass over the ring
                // (phase ph ^ 1), the others in the pass before.
                for (uint32_t k = 0; k < (uint32_t)T::stages; ++k) {
                    const uint32_t par = k < s ? ph ^ 1u : ph;
                    for (uint32_t n = 0; n < kGemmSpin && !mbar_try_wait(&bars.full[k], par); ++n)
                        ;
                }
            }
        }
    } else if (warp == kEpiWarps + 1) {              // product
        if (lane == 0) {
            constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(BN / 8) << 17) | ((128u / 16u) << 24);
            uint32_t s = 0, ph = 0, d = 0, dph = 1;
            bool ok = true;
            for (uint32_t i = blockIdx.x; i < ntile && ok; i += gridDim.x)
                for (uint32_t kb = 0; kb < p.KB; ++kb) {
                    if (!(ok = wait_bar(&bars.tempty[d], dph, bars, p.status) &&
                               wait_bar(&bars.full[s], ph, bars, p.status)))
                        break;
                    fence_after();
                    const uint32_t at = smem_addr(smem + s * T::bytes);
                    const uint64_t da = operand_desc(at), db = operand_desc(at + 128 * 128);
#pragma unroll
                    for (int k = 0; k < 4; ++k)      // 32 values: 32 bytes along the row
                        umma(tmem + d * BN, da + k * 2, db + k * 2, idesc, k > 0);
                    umma_commit(&bars.empty[s]);
                    umma_commit(&bars.tfull[d]);
                    if (++s == T::stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                    if (++d == T::bufs) {
                        d = 0;
                        dph ^= 1u;
                    }
                }
            if (!ok) {                               // products in flight
                umma_commit(&bars.drain);
                for (uint32_t n = 0; n < kGemmSpin && !mbar_try_wait(&bars.drain, 0); ++n)
                    ;
            }
        }
    } else if (warp == kEpiWarps + 2) {              // scales
        uint32_t d = 0, dph = 1;
        bool ok = true;
        for (uint32_t i = blockIdx.x; i < ntile && ok; i += gridDim.x) {
            uint32_t m, n;
            tile_at(p, i, m, n);
            const uint32_t row = m * 128u + lane, cb = (n * BN + (lane & 3u) * T::cols) >> 7;
            const float *sa = p.sa + (uint64_t)row * p.KB, *sb = p.sb + (uint64_t)cb * p.KB;
            const bool col = lane < 4u && n * BN + lane * T::cols < p.N;
            float v[4], w;
            auto load = [&](uint32_t kb) {
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j)
                    v[j] = row + j * 32u < p.M ? __ldg(sa + j * 32ull * p.KB + kb) : 0.0f;
                w = col ? __ldg(sb + kb) : 0.0f;
            };
            load(0);
            for (uint32_t kb = 0; kb < p.KB; ++kb) {
                if (!(ok = __all_sync(0xFFFFFFFFu, wait_bar(&bars.tempty[d], dph, bars, p.status))))
                    break;
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j)
                    srow[d][j * 32u + lane] = v[j];
                if (lane < 4u)
                    scol[d][lane] = w;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bars.tfull[d]);
                if (kb + 1 < p.KB)
                    load(kb + 1);
                if (++d == T::bufs) {
                    d = 0;
                    dph ^= 1u;
                }
            }
        }
    } else if (warp < kEpiWarps) {                   // sums
        const uint32_t quad = warp & 3u, part = warp >> 2;
        const uint32_t taddr = tmem + ((quad * 32u) << 16) + part * T::cols;
        char *buf = smem + T::stages * T::bytes + warp * kStageOut;
        uint32_t d = 0, dph = 0;
        bool ok = true;
        for (uint32_t i = blockIdx.x; i < ntile && ok; i += gridDim.x) {
            uint32_t m, n;
            tile_at(p, i, m, n);
            float2 acc[T::cols / 2];
#pragma unroll
            for (int j = 0; j < T::cols / 2; ++j)
                acc[j] = make_float2(0.0f, 0.0f);
            for (uint32_t kb = 0; kb < p.KB; ++kb) {
                if (!(ok = __all_sync(0xFFFFFFFFu, wait_bar(&bars.tfull[d], dph, bars, p.status))))
                    break;
                fence_after();
                const float s = srow[d][quad * 32u + lane] * scol[d][part];
                const float2 ss = make_float2(s, s);
#pragma unroll
                for (int j = 0; j < T::cols; j += 16) {
                    uint32_t v[16];
                    tmem_ld16(taddr + d * BN + j, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        acc[j / 2 + q] = __ffma2_rn(make_float2(__uint_as_float(v[2 * q]), __uint_as_float(v[2 * q + 1])),
                                                    ss, acc[j / 2 + q]);
                }
                fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bars.tempty[d]);
                if (++d == T::bufs) {
                    d = 0;
                    dph ^= 1u;
                }
            }
            if (ok)
                store_rows<T::cols, Out>(acc, buf, static_cast<Out *>(p.c), m * 128u + quad * 32u,
                                         n * BN + part * T::cols, p, lane);
        }
    }
    fence_before();
    __syncthreads();
    if (warp == kEpiWarps + 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(T::bufs * BN));
    }
}

namespace {

template <int BN, typename Out>
cudaError_t run_tile(const GemmArgs &g, int sms, cudaStream_t s)
{
    using T = Tile<BN>;
    CUtensorMap ma, mb;
    if (!make_byte_map(&ma, g.a, (uint64_t)g.M, (uint64_t)g.K, 128) ||
        !make_byte_map(&mb, g.b, (uint64_t)g.N, (uint64_t)g.K, BN))
        return cudaErrorInvalidValue;
    TileArgs p;
    p.sa = g.sa;
    p.sb = g.sb;
    p.c = g.c;
    p.status = g.status;
    p.M = (uint32_t)g.M;
    p.N = (uint32_t)g.N;
    p.K = (uint32_t)g.K;
    p.KB = (p.K + 127) / 128;
    p.mt = (p.M + 127) / 128;
    p.nt = (p.N + BN - 1) / BN;
    // a group's part of b: at most 32 MB, a quarter of L2
    const uint64_t fit = (32ull << 20) / ((uint64_t)BN * (p.K + 1)) + 1;
    p.group = fit < p.nt ? (uint32_t)fit : p.nt;
    const size_t smem = (size_t)T::stages * T::bytes + kEpiWarps * kStageOut + 1024;
    const auto k = gemm_tile_kernel<BN, Out>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess)
        return e;
    const uint64_t tiles = (uint64_t)p.mt * p.nt;
    k<<<(unsigned)(tiles < (uint64_t)sms ? tiles : sms), kTileThreads, smem, s>>>(ma, mb, p);
    return cudaGetLastError();
}

template <int NT, typename Out>
cudaError_t run_small(const GemmArgs &g, cudaStream_t s)
{
    const dim3 grid((unsigned)((g.N + 15) / 16), (unsigned)((g.M + 8 * NT - 1) / (8 * NT)));
    gemm_small_kernel<NT, Out><<<grid, 256, 0, s>>>(g.a, g.sa, g.b, g.sb, (uint32_t)g.M, (uint32_t)g.N,
                                                    (uint32_t)g.K, static_cast<Out *>(g.c));
    return cudaGetLastError();
}

template <typename Out>
cudaError_t gemm(const GemmArgs &g, cudaStream_t s)
{
    if (g.M <= kSmallM) {
        if (g.M <= 8)
            return run_small<1, Out>(g, s);
        if (g.M <= 16)
            return run_small<2, Out>(g, s);
        return run_small<4, Out>(g, s);
    }
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return e;
    // Tile width: the fewest column-steps of work on the busiest SM.  A
    // narrower tile fetches a more often, so its step is priced up.
    const int64_t mt = (g.M + 127) / 128;
    int best = 256;
    double cost = 0;
    for (int bn = 256; bn >= 64; bn /= 2) {
        const int64_t tiles = mt * ((g.N + bn - 1) / bn), rounds = (tiles + sms - 1) / sms;
        const double c = (double)rounds * (bn + 32);
        if (bn == 256 || c < cost) {
            cost = c;
            best = bn;
        }
    }
    return best == 256 ? run_tile<256, Out>(g, sms, s)
                       : best == 128 ? run_tile<128, Out>(g, sms, s) : run_tile<64, Out>(g, sms, s);
}

} // namespace

cudaError_t launch_gemm_fp8(const GemmArgs &g, int out_f32, cudaStream_t s)
{
    return out_f32 ? gemm<float>(g, s) : gemm<__nv_bfloat16>(g, s);
}

} // namespace mxq
