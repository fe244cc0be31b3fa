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
// gemm_tile_kernel (more rows).  One persistent CTA per SM, tiles of 128
// rows by BN columns.  A producer warp fetches the 128-byte-wide K blocks of a
// and b by TMA (128-byte swizzle; rows, columns and a last K block past the ends
// arrive as zeros), another issues tcgen05.mma kind::f8f6f4 (four of K = 32 a
// block) into one of several TMEM buffers, and 8 warps move each finished buffer
// into their sums: acc += (sa sb) P.  A warp has 32 rows (its TMEM lanes) and
// BN / 2 columns, so all of a thread's sums share one row scale and one column
// scale.  Two more warps bring the scales of each block into shared memory, four
// blocks ahead: loaded by the summing warps themselves, 32 lines a load, they
// took 17 % more time.  The service warps hand most of their registers to the
// summing ones (setmaxnreg), whose 128 sums a thread leave room to read one part
// of a buffer while the part before is added.  What bounds it: the sums.  At
// 65536 x 2560 x 2048 (bf16) it takes 328 us in a burst (2.1 PFLOP/s), 370 to 390
// under the power limit; the same products and copies without sums and stores take
// 224.
//
// gemm_small_kernel (few rows: decoding).  The read of b is the bound.  A
// warp multiplies 16 rows of b by up to 8 NT rows of a with mma.sync
// m16n8k32; 8 or 16 warps of a CTA split K by blocks and add their sums in a fixed
// order (1 x 2560 x 2048 2.4 us).  Both operands come straight from global memory: a lane's 16-byte
// pieces of a row of b and of a row of a hold the same k, and the order of k
// inside a block is free.
//
// Scales far out.  sa sb is formed in fp32 and may leave its range where sa sb P does
// not.  No sum pays for that: the streamed ones are formed in a range of their own
// (kLift), and for the tiles the warps that bring the scales keep the smallest and the
// largest of an item; where a product may leave the range the item's sums are formed
// again from global memory (sum_far).  A choice at every step, by the summing warps, took
// 4 to 8 % more time at 65536 x 2560 x 2048, by either way that was tried.
//
// Every wait is bounded: a wait that runs into its limit sets
// MXQ_DEV_WAIT_TIMEOUT and all roles leave their loops.  The producer and the product
// warp leave theirs, on that way and on the ordinary one, behind the last of what
// they have started (bounded waits too): whichever role gives up, and when, no
// copy or product is in flight where TMEM is freed and the CTA ends.
#include "mxq_cluster.cuh"
#include "mxq_device.cuh"
#include "mxq_internal.h"
#include "mxq.h"
#include "mxq_test.h"
#include "mxq_tcgen05.cuh"
#include "mxq_tma.cuh"
#include <algorithm>
#include <atomic>

namespace mxq {

namespace {

// Waits give up after this many tests; a test suspends for 4 us at most (measured),
// so after a second (65 ms in a launch that was told to stall).  A wait that makes
// progress takes up to some ms, where the sums of an item are formed again.
constexpr uint32_t kGemmSpin = 1u << 18, kStalledSpin = 1u << 14;

// Test hook (include/mxq_test.h): the next launch of tiles stalls on purpose.
std::atomic<int> g_stall_product{0};

// Rows that stream b through mma.sync: up to 16, and more while the whole product
// (with K counted as 1024 at least, a block a warp) is small.  Measured, tiles against streaming: 16 x 2560 x 2048 6.5 against
// 3.4 us, 20 rows of it (0.1 G) 6.5 against 8.5; 20 x 1999 x 1552 (62 M) 7.5 against
// 4.6, 33 x 2048 x 1280 (87 M) 5.0 against 7.2; 128 x 512 x 512 4.2 against 2.9; of
// short rows 496 x 4567 x 16 5.6 against 47.6.
// (At most 1024 rows of it, far inside the grid's second dimension.)
constexpr int64_t kSmallM = 16, kSmallMaxM = 1024, kSmallWork = 64 << 20;

template <typename T>
__device__ __forceinline__ T to_out(float v);
template <>
__device__ __forceinline__ float to_out<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 to_out<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Factor f of a block's sum P from its two scales: f = a b.  Where that leaves the
// normal numbers although neither scale is 0, Inf or NaN, the scaled sum may still be
// in range (|P| is 0 or from 2^-18 to below 2^25); (P pre) f is formed instead.  Of
// scales whose product underflows pre is the larger one (P pre overflows only if the
// smaller were 0), of scales whose product overflows the smaller one, which is above
// 1 (P pre overflows only if P a b does).
__device__ __forceinline__ void split_scales(float a, float b, float &f, float &pre)
{
    f = a * b;
    pre = 1.0f;
    const uint32_t e = __float_as_uint(f) & 0x7F800000u;
    if ((e == 0u || e == 0x7F800000u) && a != 0.0f && b != 0.0f && fabsf(a) < INFINITY && fabsf(b) < INFINITY) {
        const bool a_first = (fabsf(a) > fabsf(b)) == (e == 0u);
        pre = a_first ? a : b;
        f = a_first ? b : a;
    }
}

// Smallest magnitude that is not 0 and largest magnitude of some scales, as twice
// their bits (less 1 for the smallest: zeros are then above everything).
struct Extremes {
    uint32_t lo = 0xFFFFFFFFu, hi = 0u;
    __device__ __forceinline__ void add(float s)
    {
        const uint32_t u = __float_as_uint(s) * 2u;
        lo = min(lo, u - 1u);
        hi = max(hi, u);
    }
    // Of the whole warp's.
    __device__ __forceinline__ void reduce()
    {
        lo = __reduce_min_sync(0xFFFFFFFFu, lo);
        hi = __reduce_max_sync(0xFFFFFFFFu, hi);
    }
    __device__ __forceinline__ float low() const { return __uint_as_float((lo >> 1) + (lo & 1u)); }
    __device__ __forceinline__ float high() const { return __uint_as_float(hi >> 1); }
};

// Whether a product of a scale of each set may leave the normal numbers.
__device__ __forceinline__ bool far_apart(const Extremes &a, const Extremes &b)
{
    const bool none = a.lo == 0xFFFFFFFFu || b.lo == 0xFFFFFFFFu;       // zeros only
    return (!none && a.low() * b.low() < 0x1p-126f) || !(a.high() * b.high() < INFINITY);
}

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

// The blocks of K from `first` on, STEP apart and below `last`: 16 rows of b from n0 on times
// 8 NT rows of a from m0 on, scaled and added up, the scales of a block kept apart where
// their product would leave the range.  acc[i][j] is row m0 + 8 i + 2 (lane % 4) + (j & 1),
// column n0 + lane / 4 + 8 (j >> 1).
template <int NT, int STEP>
__device__ __forceinline__ void split_blocks(const uint8_t *__restrict__ a, const float *__restrict__ sa,
                                             const uint8_t *__restrict__ b, const float *__restrict__ sb, uint32_t M,
                                             uint32_t N, uint32_t K, uint32_t m0, uint32_t n0, uint32_t first,
                                             uint32_t last, uint32_t lane, float (&acc)[NT][4])
{
    const uint32_t g = lane >> 2, t = lane & 3u, KB = (K + 127u) / 128u;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const bool r0 = n0 + g < N, r1 = n0 + g + 8u < N;
    const uint8_t *b0 = b + (uint64_t)(n0 + g) * K, *b1 = b0 + 8ull * K;
#pragma unroll
    for (int i = 0; i < NT; ++i)
        acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
#pragma unroll 1
    for (uint32_t kb = first; kb < last; kb += STEP) {
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
            float f0, f1, pre0, pre1;
            split_scales(mc < M ? __ldg(sa + (uint64_t)mc * KB + kb) : 0.0f, wb, f0, pre0);
            split_scales(mc + 1u < M ? __ldg(sa + (uint64_t)(mc + 1u) * KB + kb) : 0.0f, wb, f1, pre1);
            float p[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma16832(p, x0.x, y0.x, x0.y, y0.y, v0.x, v0.y);
            mma16832(p, x0.z, y0.z, x0.w, y0.w, v0.z, v0.w);
            mma16832(p, x1.x, y1.x, x1.y, y1.y, v1.x, v1.y);
            mma16832(p, x1.z, y1.z, x1.w, y1.w, v1.z, v1.w);
            acc[i][0] = fmaf(p[0] * pre0, f0, acc[i][0]);
            acc[i][1] = fmaf(p[1] * pre1, f1, acc[i][1]);
            acc[i][2] = fmaf(p[2] * pre0, f0, acc[i][2]);
            acc[i][3] = fmaf(p[3] * pre1, f1, acc[i][3]);
        }
    }
}

// The streamed sums are formed times 2^64 and brought back at the end: a product of
// two scales that underflows all the same (below 2^-190) adds less than 2^-165, nothing in
// fp32.  One that overflows leaves Inf or NaN in a warp's part of a sum, and the CTA's sums
// are formed again; so they are where a part reaches kFar, since up to 16 of them are added.
constexpr float kLift = 0x1p64f, kFar = 0x1p120f;

// The warps' parts of the CTA's sums, added up in their order and brought back by `unit`, to c.
template <int NT, int W, typename Out>
__device__ __forceinline__ void store_streamed(const float (*red)[NT * 8][17], float unit, uint32_t M, uint32_t N,
                                               uint32_t m0, uint32_t n0, Out *c)
{
    for (uint32_t i = threadIdx.x; i < NT * 128u; i += 32u * W) {
        const uint32_t m = i >> 4, n = i & 15u;
        float s = red[0][m][n];
#pragma unroll
        for (int w = 1; w < W; ++w)
            s += red[w][m][n];
        if (m0 + m < M && n0 + n < N)
            c[(uint64_t)(m0 + m) * N + n0 + n] = to_out<Out>(s * unit);
    }
}

// The CTA's sums once more, with the scales kept apart.  Out of line: a call that is hardly
// ever made costs the kernel no registers.
template <int NT, int W, typename Out>
__device__ __noinline__ void stream_again(const uint8_t *a, const float *sa, const uint8_t *b, const float *sb, uint32_t M,
                                          uint32_t N, uint32_t K, float (*red)[NT * 8][17], Out *c)
{
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3u;
    const uint32_t n0 = blockIdx.x * 16u, m0 = blockIdx.y * (8u * NT);
    float acc[NT][4];
    split_blocks<NT, W>(a, sa, b, sb, M, N, K, m0, n0, warp, (K + 127u) / 128u, lane, acc);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            red[warp][i * 8 + t * 2 + (j & 1)][g + (j >> 1) * 8] = acc[i][j];
    __syncthreads();
    store_streamed<NT, W>(red, 1.0f, M, N, m0, n0, c);
}

// Up to 8 rows: 1024 threads an SM (with fewer, 1 x 2560 x 2048 takes a second round of CTAs).
template <int NT, int W, typename Out>
__global__ void __launch_bounds__(32 * W, NT == 1 ? 32 / W : 0)
gemm_small_kernel(const uint8_t *__restrict__ a, const float *__restrict__ sa, const uint8_t *__restrict__ b,
                  const float *__restrict__ sb, uint32_t M, uint32_t N, uint32_t K, Out *__restrict__ c)
{
    __shared__ float red[W][NT * 8][17];
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3u;
    const uint32_t n0 = blockIdx.x * 16u, m0 = blockIdx.y * (8u * NT), KB = (K + 127u) / 128u;
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const bool r0 = n0 + g < N, r1 = n0 + g + 8u < N;
    const uint8_t *b0 = b + (uint64_t)(n0 + g) * K, *b1 = b0 + 8ull * K;
    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
        acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
#pragma unroll 2
    for (uint32_t kb = warp; kb < KB; kb += W) {
        const uint32_t k0 = kb * 128u + t * 16u, k1 = k0 + 64u;
        const bool p0 = k0 < K, p1 = k1 < K;
        const uint4 x0 = r0 && p0 ? __ldg(reinterpret_cast<const uint4 *>(b0 + k0)) : zero;
        const uint4 x1 = r0 && p1 ? __ldg(reinterpret_cast<const uint4 *>(b0 + k1)) : zero;
        const uint4 y0 = r1 && p0 ? __ldg(reinterpret_cast<const uint4 *>(b1 + k0)) : zero;
        const uint4 y1 = r1 && p1 ? __ldg(reinterpret_cast<const uint4 *>(b1 + k1)) : zero;
        const float wb = __ldg(sb + (uint64_t)(n0 >> 7) * KB + kb) * kLift;
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
    bool far = false;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            far |= !(fabsf(acc[i][j]) < kFar);
    if (__syncthreads_or(far))
        stream_again<NT, W>(a, sa, b, sb, M, N, K, red, c);
    else
        store_streamed<NT, W>(red, 1.0f / kLift, M, N, m0, n0, c);
}

// ------------------------------------------------------------ many rows --

constexpr int kEpiWarps = 8;
constexpr int kTileThreads = 32 * (kEpiWarps + 4);   // sums, producer, product, two of scales
// Registers of a thread: kTileThreads x 168 at launch (what __launch_bounds__
// allows), of which the four service warps give up the most.  The sum of the
// shares must not pass what the block was launched with.
constexpr int kLaunchRegs = 168, kSumRegs = 232, kServiceRegs = 40;
static_assert(kEpiWarps * kSumRegs + 4 * kServiceRegs <= (kEpiWarps + 4) * kLaunchRegs, "register shares");
constexpr uint32_t kBoxB = 64;                       // rows of a copy of b
constexpr int kStageOut = 4096;                      // bytes a warp stages its result through

template <int BN>
struct Tile {
    static constexpr int bytes = (128 + BN) * 128;                    // one K block of a and b
    static constexpr int stages = BN == 256 ? 4 : BN == 128 ? 5 : 7;  // 227 KB in all
    static constexpr int bufs = BN == 256 ? 2 : 4;                    // TMEM buffers of BN columns
};

struct TileArgs {
    const uint8_t *a, *b;
    const float *sa, *sb;
    void *c;
    uint32_t *status;
    uint32_t M, N, K, KB;
    uint32_t mt, nt;            // tiles in each direction
    uint32_t group;             // column tiles of a group; groups are walked one after the other
    uint32_t whole, cut;        // tiles after the first `whole` are cut into 2^cut parts of their columns
    uint32_t items;             // whole tiles and parts
    uint32_t tma_out;           // c is stored by TMA (rows of a multiple of 16 bytes)
    uint32_t spin;              // tests of a barrier before a wait gives up
    uint32_t stall;             // test hook: 1, 2: the scales of CTA 0's first, last step are never reported
};

// Items whose flags of far scales are kept: more than the scale warps run ahead, which
// is by one step a buffer.
constexpr uint32_t kFarRing = 8;

struct TileBars {
    uint64_t full[8], empty[8], tfull[4], tempty[4], drain;
    uint32_t tmem, abort;
    uint32_t far[2][kFarRing];      // by half of the rows and item: scales whose products may leave the range
};

// Item number -> its first row and column and its width, a whole tile of BN
// columns or a part.  Inside a group of column tiles the columns run fastest, so
// that the rows of a that the CTAs share at a time are few and the group's part
// of b stays in L2.
template <int BN>
__device__ __forceinline__ void item_at(const TileArgs &p, uint32_t i, uint32_t &m0, uint32_t &n0, uint32_t &width)
{
    uint32_t tile = i, part = 0;
    width = BN;
    if (BN == 256 && i >= p.whole) {
        tile = p.whole + ((i - p.whole) >> p.cut);
        width = BN >> p.cut;
        part = (i - p.whole) & ((1u << p.cut) - 1u);
    }
    const uint32_t per = p.mt * p.group, grp = tile / per, in = tile - grp * per;
    const uint32_t w = min(p.group, p.nt - grp * p.group), m = in / w;
    m0 = m * 128u;
    n0 = (grp * p.group + (in - m * w)) * BN + part * width;
}

__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, TileBars &s, const TileArgs &p)
{
    for (uint32_t i = 0; i < p.spin; ++i) {
        if (mbar_try_wait(bar, parity))
            return true;
        if ((i & 63u) == 63u && *reinterpret_cast<volatile uint32_t *>(&s.abort))
            return false;
    }
    *reinterpret_cast<volatile uint32_t *>(&s.abort) = 1u;
    atomicOr(p.status, MXQ_DEV_WAIT_TIMEOUT);
    return false;
}

// The same for a role that leaves: it waits whether or not another one gave up.
__device__ __forceinline__ void wait_out(uint64_t *bar, uint32_t parity)
{
    for (uint32_t i = 0; i < kGemmSpin && !mbar_try_wait(bar, parity); ++i)
        ;
}

// The instructions below are issued by the lane whose `one` is 1, inside code
// that the whole warp runs: their descriptors and addresses then stay in
// uniform registers.  In a branch of one thread each product took 85 cycles to
// issue, and a step of four with its commits 710 cycles instead of 512.
__device__ __forceinline__ void umma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add, uint32_t one)
{
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "setp.ne.u32 p, %4, 0;\n\t"
                 "setp.ne.u32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"(one) : "memory");
}

__device__ __forceinline__ void expect_tx(uint64_t *bar, uint32_t bytes, uint32_t one)
{
    asm volatile("{\n\t.reg .pred q;\n\t"
                 "setp.ne.u32 q, %2, 0;\n\t"
                 "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}"
                 ::"r"(smem_addr(bar)), "r"(bytes), "r"(one) : "memory");
}

__device__ __forceinline__ void tma_load(void *dst, const CUtensorMap *map, uint32_t x, uint32_t y, uint64_t *bar,
                                         uint32_t one)
{
    asm volatile("{\n\t.reg .pred q;\n\t"
                 "setp.ne.u32 q, %5, 0;\n\t"
                 "@q cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%3, %4}], [%2];\n\t}"
                 ::"r"(smem_addr(dst)), "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(one) : "memory");
}

// Sums of 16 bytes' worth of results -> their bits.
template <typename Out>
__device__ __forceinline__ uint4 out_bits(const float2 *s)
{
    if constexpr (sizeof(Out) == 4)
        return make_uint4(__float_as_uint(s[0].x), __float_as_uint(s[0].y), __float_as_uint(s[1].x),
                          __float_as_uint(s[1].y));
    else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(s[i].x, s[i].y);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// One warp's 32 rows x COLS sums -> global by TMA: 128 bytes of each row at a
// time, through 4 KB of shared memory in the map's swizzle.  The copy reads them
// while the warp goes on; the next one waits for that.  Rows and columns past
// the ends are left out by the copy.
template <int COLS, typename Out>
__device__ __forceinline__ void store_tma(const float2 *acc, char *buf, const CUtensorMap *map, uint32_t m0,
                                          uint32_t n0, const TileArgs &p, uint32_t lane)
{
    constexpr int per = 128 / sizeof(Out);      // columns of a copy
    constexpr int used = COLS < per ? COLS : per;
#pragma unroll
    for (int r = 0; r < COLS / used; ++r) {
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
#pragma unroll
        for (int q = 0; q < used * (int)sizeof(Out) / 16; ++q)
            *reinterpret_cast<uint4 *>(buf + lane * 128u + (((uint32_t)q ^ (lane & 7u)) << 4)) =
                out_bits<Out>(acc + (r * used + q * (16 / (int)sizeof(Out))) / 2);
        fence_proxy_async_smem();
        __syncwarp();
        const uint32_t n = n0 + r * used;
        if (lane == 0 && m0 < p.M && n < p.N)
            asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];"
                         ::"l"(map), "r"(smem_addr(buf)), "r"(n), "r"(m0) : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
}

// The same by plain stores, for rows that are no multiple of 16 bytes and for
// warps of less than 128 bytes a row: up to 128 bytes of each row at a time, their
// 16-byte pieces permuted against bank conflicts, written out along the rows.
template <int COLS, typename Out>
__device__ __forceinline__ void store_rows(const float2 *acc, char *buf, Out *c, uint32_t m0, uint32_t n0,
                                           const TileArgs &p, uint32_t lane)
{
    constexpr int per = 128 / sizeof(Out);      // columns a round
    constexpr int used = COLS < per ? COLS : per;
    constexpr int pieces = used * (int)sizeof(Out) / 16;
#pragma unroll
    for (int r = 0; r < COLS / used; ++r) {
        __syncwarp();
#pragma unroll
        for (int q = 0; q < pieces; ++q)
            *reinterpret_cast<uint4 *>(buf + lane * 128u + (((uint32_t)q ^ (lane & 7u)) << 4)) =
                out_bits<Out>(acc + (r * used + q * (16 / (int)sizeof(Out))) / 2);
        __syncwarp();
        const uint32_t nr = n0 + r * used;
        if (p.tma_out) {        // whole pieces
            constexpr int rows = 32 / pieces;
#pragma unroll
            for (int i = 0; i < pieces; ++i) {
                const uint32_t row = i * rows + lane / pieces, q = lane % pieces, n = nr + q * (16u / sizeof(Out));
                if (m0 + row < p.M && n < p.N)
                    *reinterpret_cast<uint4 *>(c + (uint64_t)(m0 + row) * p.N + n) =
                        *reinterpret_cast<const uint4 *>(buf + row * 128u + ((q ^ (row & 7u)) << 4));
            }
            continue;
        }
        if (sizeof(Out) == 2 && (p.N & 1u) == 0) {      // two at a time
            constexpr int lanes = used / 2, rows = 32 / lanes;
            const uint32_t col = (lane % lanes) * 2u, sub = lane / lanes;
            Out *o = c + (uint64_t)(m0 + sub) * p.N + nr + col;
#pragma unroll 16
            for (int i = 0; i < 32 / rows; ++i, o += (uint64_t)rows * p.N) {
                const uint32_t row = i * rows + sub, at = col * 2u;
                if (m0 + row < p.M && nr + col < p.N)
                    *reinterpret_cast<uint32_t *>(o) = *reinterpret_cast<const uint32_t *>(
                        buf + row * 128u + (((at >> 4) ^ (row & 7u)) << 4) + (at & 15u));
            }
            continue;
        }
        // element by element: a lane has a column (or two, 32 apart), and rows follow one another
        constexpr int lanes = used < 32 ? used : 32, rows = 32 / lanes;
        const uint32_t col = lane % lanes, sub = lane / lanes;
        Out *o = c + (uint64_t)(m0 + sub) * p.N + nr + col;
        constexpr int ahead = sizeof(Out) == 4 ? 32 : 16;      // 8192 x 1999 x 1552: fp32 46 us (with 16 55), bf16 39
#pragma unroll ahead
        for (int i = 0; i < 32 / rows; ++i, o += (uint64_t)rows * p.N) {
            const uint32_t row = i * rows + sub;
#pragma unroll
            for (int k = 0; k < used; k += lanes) {
                const uint32_t at = (col + k) * (uint32_t)sizeof(Out);
                if (m0 + row < p.M && nr + col + k < p.N)
                    o[k] = *reinterpret_cast<const Out *>(buf + row * 128u + (((at >> 4) ^ (row & 7u)) << 4) + (at & 15u));
            }
        }
    }
}

// A summing warp's part of an item of W columns, its 32 rows and W / 2 columns:
// the scaled sum of `steps` products that come through the TMEM buffers d,
// d + 1, ... of BN columns.
template <int W, int BN>
__device__ __forceinline__ bool sum_steps(const TileArgs &p, TileBars &bars, const float (*srow)[128],
                                          const float (*scol)[2], uint32_t tmem, uint32_t steps, uint32_t warp,
                                          uint32_t lane, uint32_t &d, uint32_t &dph, float2 (&acc)[W / 4])
{
    constexpr int cols = W / 2;
    const uint32_t quad = warp & 3u, part = warp >> 2;
    const uint32_t taddr = tmem + ((quad * 32u) << 16) + part * cols;
    const float *const rows = &srow[0][quad * 32u + lane], *const col = &scol[0][part];
#pragma unroll
    for (int j = 0; j < cols / 2; ++j)
        acc[j] = make_float2(0.0f, 0.0f);
    for (uint32_t kb = 0; kb < steps; ++kb) {
        if (!__all_sync(0xFFFFFFFFu, wait_bar(&bars.tfull[d], dph, bars, p)))
            return false;
        fence_after();
        const float f = rows[d * 128u] * col[d * 2u];
        const float2 ff = make_float2(f, f);
        const uint32_t at = taddr + d * BN;
        uint32_t v[2][32];
        tmem_ld32(at, v[0]);
        tmem_ld_wait(v[0]);
#pragma unroll
        for (int j = 0; j < cols / 32; ++j) {
            uint32_t(&now)[32] = v[j & 1], (&next)[32] = v[(j + 1) & 1];
            if ((j + 1) * 32 < cols)
                tmem_ld32(at + (j + 1) * 32, next);
            else {                           // all of the buffer is read
                fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bars.tempty[d]);
            }
#pragma unroll
            for (int q = 0; q < 16; ++q)
                acc[j * 16 + q] = __ffma2_rn(make_float2(__uint_as_float(now[2 * q]), __uint_as_float(now[2 * q + 1])),
                                             ff, acc[j * 16 + q]);
            if ((j + 1) * 32 < cols)
                tmem_ld_wait(next);
        }
        if (++d == Tile<BN>::bufs) {
            d = 0;
            dph ^= 1u;
        }
    }
    return true;
}

// COLS columns of this warp's 32 rows from (m0, n0) on -> c.
template <int COLS, typename Out>
__device__ __forceinline__ void store_sums(const float2 *acc, char *buf, const CUtensorMap *mc, uint32_t m0,
                                           uint32_t n0, const TileArgs &p, uint32_t lane)
{
    if (p.tma_out && COLS * sizeof(Out) >= 128)
        store_tma<COLS, Out>(acc, buf, mc, m0, n0, p, lane);
    else {
        // a copy of an item before may still read the buffer
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        store_rows<COLS, Out>(acc, buf, static_cast<Out *>(p.c), m0, n0, p, lane);
    }
}

// Whether a summing warp's item (the CTA's `item`-th, all of its steps read) has scales far out.
__device__ __forceinline__ bool far_item(const TileBars &bars, uint32_t warp, uint32_t item)
{
    return __any_sync(0xFFFFFFFFu, bars.far[(warp & 3u) >> 1][item % kFarRing] != 0u);
}

// The sums of a warp's 32 rows and `cols` columns from (m0, n0) on over the K blocks
// [k0, k1) once more, from global memory, with the scales of a block kept apart: for
// items with scales far out, which take about ten times as long.  To c, or
// (SHARE) to the partial sums [column / 4][row] of a cluster.
template <typename Out, bool SHARE>
__device__ __forceinline__ void sum_far(const TileArgs &p, void *dst, uint32_t m0, uint32_t n0, uint32_t cols, uint32_t k0,
                                     uint32_t k1, uint32_t lane)
{
    for (uint32_t n = 0; n < cols; n += 16u) {
        float acc[4][4];
        split_blocks<4, 1>(p.a, p.sa, p.b, p.sb, p.M, p.N, p.K, m0, n0 + n, k0, n0 + n < p.N ? k1 : k0, lane, acc);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t row = i * 8u + (lane & 3u) * 2u + (j & 1), col = n + (lane >> 2) + (j >> 1) * 8u;
                if (SHARE)
                    static_cast<float *>(dst)[(col >> 2) * 512u + row * 4u + (col & 3u)] = acc[i][j];
                else if (m0 + row < p.M && n0 + col < p.N)
                    static_cast<Out *>(dst)[(uint64_t)(m0 + row) * p.N + n0 + col] = to_out<Out>(acc[i][j]);
            }
    }
}

template <int W, int BN, typename Out>
__device__ __forceinline__ bool sum_item(const TileArgs &p, const CUtensorMap *mc, TileBars &bars,
                                         const float (*srow)[128], const float (*scol)[2], uint32_t tmem, char *buf,
                                         uint32_t m0, uint32_t n0, uint32_t warp, uint32_t lane, uint32_t &d,
                                         uint32_t &dph, uint32_t item)
{
    float2 acc[W / 4];
    if (!sum_steps<W, BN>(p, bars, srow, scol, tmem, p.KB, warp, lane, d, dph, acc))
        return false;
    m0 += (warp & 3u) * 32u;
    n0 += (warp >> 2) * (W / 2);
    if (far_item(bars, warp, item))
        sum_far<Out, false>(p, p.c, m0, n0, W / 2, 0, p.KB, lane);
    else
        store_sums<W / 2, Out>(acc, buf, mc, m0, n0, p, lane);
    return true;
}

} // namespace

// S > 1: a cluster of S CTAs shares an item (the grid holds S CTAs an item), each
// over its part of K; their sums meet in shared memory, where each CTA adds up a
// part of the columns in the order of the CTAs.
template <int BN, typename Out, int S>
__global__ void __launch_bounds__(kTileThreads, 1)
gemm_tile_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                 const __grid_constant__ CUtensorMap mc, const TileArgs p)
{
    using T = Tile<BN>;
    constexpr int kCols = T::bufs * BN;      // TMEM columns: 256 or 512
    extern __shared__ __align__(1024) char smem_raw[];
    __shared__ TileBars bars;
    __shared__ float srow[T::bufs][128], scol[T::bufs][2];
    // operand tiles start on 1024-byte boundaries (the swizzle repeats there)
    char *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    // the same value in every lane, and known to be
    const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31u;
    const uint32_t rank = blockIdx.x % S, item0 = blockIdx.x / S, items_on = gridDim.x / S;
    const uint32_t k0 = p.KB * rank / S, k1 = p.KB * (rank + 1u) / S;      // this CTA's K blocks
    if (threadIdx.x == 0) {
        for (int i = 0; i < T::stages; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < T::bufs; ++i) {
            mbar_init(&bars.tfull[i], 3);            // the product and two warps' scales
            mbar_init(&bars.tempty[i], kEpiWarps);
        }
        mbar_init(&bars.drain, 1);
        bars.abort = 0;
        fence_mbar_init();
    }
    if (warp == kEpiWarps + 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_addr(&bars.tmem)), "n"(kCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = bars.tmem;
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();

    if (warp >= kEpiWarps) {
        regs_down<kServiceRegs>();
        if (warp == kEpiWarps) {                     // producer
            const uint32_t one = elect_one();
            uint32_t s = 0, ph = 1;                  // a fresh barrier passes the wait for its odd phase
            bool ok = true;
            for (uint32_t i = item0; i < p.items && ok; i += items_on) {
                uint32_t m0, n0, w;
                item_at<BN>(p, i, m0, n0, w);
                for (uint32_t kb = k0; kb < k1; ++kb) {
                    if (!(ok = __all_sync(0xFFFFFFFFu, wait_bar(&bars.empty[s], ph, bars, p))))
                        break;
                    char *dst = smem + s * T::bytes;
                    expect_tx(&bars.full[s], (128u + w) * 128u, one);
                    tma_load(dst, &ma, kb * 128u, m0, &bars.full[s], one);
#pragma unroll
                    for (uint32_t r = 0; r < BN; r += kBoxB)
                        if (r < w)
                            tma_load(dst + (128u + r) * 128u, &mb, kb * 128u, n0 + r, &bars.full[s], one);
                    if (++s == T::stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            // The last fill of every stage has landed.  Stages before s were filled in the
            // current pass over the ring (phase ph ^ 1), the others in the pass before
            // (a stage never filled passes the wait for its odd phase).
            for (uint32_t k = 0; k < (uint32_t)T::stages; ++k)
                wait_out(&bars.full[k], k < s ? ph ^ 1u : ph);
        } else if (warp == kEpiWarps + 1) {          // product
            const uint32_t one = elect_one();
            uint32_t s = 0, ph = 0, d = 0, dph = 1;
            bool ok = true;
            for (uint32_t i = item0; i < p.items && ok; i += items_on) {
                const uint32_t w = BN == 256 && i >= p.whole ? BN >> p.cut : BN;
                const uint32_t idesc = (1u << 4) | ((w / 8u) << 17) | ((128u / 16u) << 24);
                for (uint32_t kb = k0; kb < k1; ++kb) {
                    ok = wait_bar(&bars.tempty[d], dph, bars, p) && wait_bar(&bars.full[s], ph, bars, p);
                    if (!(ok = __all_sync(0xFFFFFFFFu, ok)))
                        break;
                    fence_after();
                    const uint32_t at = smem_addr(smem + s * T::bytes);
                    const uint64_t da = operand_desc(at), db = operand_desc(at + 128 * 128);
#pragma unroll
                    for (int k = 0; k < 4; ++k)      // 32 values: 32 bytes along the row
                        umma(tmem + d * BN, da + k * 2, db + k * 2, idesc, k > 0, one);
                    umma_commit(&bars.tfull[d], one);
                    umma_commit(&bars.empty[s], one);
                    if (++s == T::stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                    if (++d == T::bufs) {
                        d = 0;
                        dph ^= 1u;
                    }
                }
            }
            umma_commit(&bars.drain, one);           // every product is done
            wait_out(&bars.drain, 0);
        } else {                                         // scales: two warps, 64 rows each
            // kAhead steps' scales at a time, and those of the steps after them on
            // the way: a load takes longer than a step.
            constexpr uint32_t kAhead = 4;
            const uint32_t sw = warp - (kEpiWarps + 2), r0 = sw * 64u + lane;
            float now[3][kAhead], next[3][kAhead];       // this lane's two rows, and (lanes 0, 1) the columns
            uint32_t d = 0, dph = 1, ni = item0, nkb = k0;    // the chunk to load next
            bool ok = true;
            auto load = [&]() {
                if (ni >= p.items)
                    return;
                uint32_t m0, n0, w;
                item_at<BN>(p, ni, m0, n0, w);
                const uint32_t row = m0 + r0, c0 = n0 + lane * (w / 2u);
                const float *sa = p.sa + (uint64_t)row * p.KB + nkb, *sb = p.sb + (uint64_t)(c0 >> 7) * p.KB + nkb;
                const bool in0 = row < p.M, in1 = row + 32u < p.M, inc = lane < 2u && c0 < p.N;
    #pragma unroll
                for (uint32_t j = 0; j < kAhead; ++j) {
                    const bool in = nkb + j < k1;
                    next[0][j] = in && in0 ? __ldg(sa + j) : 0.0f;
                    next[1][j] = in && in1 ? __ldg(sa + 32ull * p.KB + j) : 0.0f;
                    next[2][j] = in && inc ? __ldg(sb + j) : 0.0f;
                }
                nkb += kAhead;
                if (nkb >= k1) {
                    nkb = k0;
                    ni += items_on;
                }
            };
            load();
            uint32_t item = 0;
            for (uint32_t i = item0; i < p.items && ok; i += items_on, ++item) {
                Extremes er, ec;                     // of the item's row and column scales
                for (uint32_t kb = k0; kb < k1 && ok; kb += kAhead) {
    #pragma unroll
                    for (uint32_t j = 0; j < kAhead; ++j) {
                        now[0][j] = next[0][j];
                        now[1][j] = next[1][j];
                        now[2][j] = next[2][j];
                    }
                    load();
    #pragma unroll
                    for (uint32_t j = 0; j < kAhead; ++j) {
                        if (kb + j >= k1 || !ok)
                            break;
                        ok = __all_sync(0xFFFFFFFFu, wait_bar(&bars.tempty[d], dph, bars, p));
                        if (!ok)
                            break;
                        srow[d][r0] = now[0][j];
                        srow[d][r0 + 32u] = now[1][j];
                        if (sw == 0 && lane < 2u)
                            scol[d][lane] = now[2][j];
                        er.add(now[0][j]);
                        er.add(now[1][j]);
                        ec.add(now[2][j]);
                        if (kb + j + 1u == k1) {
                            er.reduce();
                            ec.reduce();
                            if (lane == 0)
                                bars.far[sw][item % kFarRing] = far_apart(er, ec);
                        }
                        __syncwarp();
                        const bool held = p.stall != 0u && blockIdx.x == 0 && sw == 0 &&
                                          (p.stall == 1u ? i == item0 && kb + j == k0
                                                         : i + items_on >= p.items && kb + j + 1u == k1);
                        if (lane == 0 && !held)
                            mbar_arrive(&bars.tfull[d]);
                        if (++d == T::bufs) {
                            d = 0;
                            dph ^= 1u;
                        }
                    }
                }
            }
        }
    } else {                                         // sums
        regs_up<kSumRegs>();
        char *buf = smem + T::stages * T::bytes + warp * kStageOut;
        uint32_t d = 0, dph = 0;
        bool ok = true;
        if constexpr (S > 1) {
            constexpr int cols = BN / 2, mine = cols / S;
            const uint32_t quad = warp & 3u, part = warp >> 2, row = quad * 32u + lane;
            uint32_t m0, n0, w;
            item_at<BN>(p, item0, m0, n0, w);
            // [part][column / 4][row], in the ring of stages
            float4 *xs = reinterpret_cast<float4 *>(smem) + part * (cols / 4) * 128u + row;
            float2 acc[cols / 2];
            ok = sum_steps<BN, BN>(p, bars, srow, scol, tmem, k1 - k0, warp, lane, d, dph, acc);
            // All steps read: the ring is empty.  After a wait that ran out it may not be, and
            // is left alone (the cluster's result is undefined then).
            if (ok && far_item(bars, warp, 0))
                sum_far<Out, true>(p, xs - lane, m0 + quad * 32u, n0 + part * cols, cols, k0, k1, lane);
            else if (ok)
#pragma unroll
                for (int q = 0; q < cols / 4; ++q)
                    xs[q * 128] = make_float4(acc[2 * q].x, acc[2 * q].y, acc[2 * q + 1].x, acc[2 * q + 1].y);
            cluster_sync_all();
            float2 sum[mine / 2];
#pragma unroll
            for (int q = 0; q < mine / 4; ++q) {
                float4 v[S];
#pragma unroll
                for (int r = 0; r < S; ++r)
                    v[r] = peer_f4(xs + (rank * (mine / 4) + q) * 128u, r);
#pragma unroll
                for (int r = 1; r < S; ++r)
                    v[0] = make_float4(v[0].x + v[r].x, v[0].y + v[r].y, v[0].z + v[r].z, v[0].w + v[r].w);
                sum[2 * q] = make_float2(v[0].x, v[0].y);
                sum[2 * q + 1] = make_float2(v[0].z, v[0].w);
            }
            if (ok)
                store_sums<mine, Out>(sum, buf, &mc, m0 + quad * 32u, n0 + part * cols + rank * mine, p, lane);
        } else for (uint32_t i = item0, item = 0; i < p.items && ok; i += items_on, ++item) {
            uint32_t m0, n0, w;
            item_at<BN>(p, i, m0, n0, w);
            if (BN < 256 || w == BN)
                ok = sum_item<BN, BN, Out>(p, &mc, bars, srow, scol, tmem, buf, m0, n0, warp, lane, d, dph, item);
            else if (w == 128)
                ok = sum_item<128, BN, Out>(p, &mc, bars, srow, scol, tmem, buf, m0, n0, warp, lane, d, dph, item);
            else
                ok = sum_item<64, BN, Out>(p, &mc, bars, srow, scol, tmem, buf, m0, n0, warp, lane, d, dph, item);
        }
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    if constexpr (S > 1) {
        if (warp >= kEpiWarps)
            cluster_sync_all();             // the sums are there (also after a wait that ran out)
        cluster_sync_all();                 // and read
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (warp == kEpiWarps + 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kCols));
    }
}

namespace {

template <int BN, typename Out, int S>
cudaError_t run_tile(const GemmArgs &g, int sms, uint32_t cut, cudaStream_t s)
{
    using T = Tile<BN>;
    TileArgs p;
    p.a = g.a;
    p.b = g.b;
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
    p.tma_out = (g.N * sizeof(Out)) % 16 == 0;
    CUtensorMap ma, mb, mc;
    if (!make_byte_map(&ma, g.a, (uint64_t)g.M, (uint64_t)g.K, 128) ||
        !make_byte_map(&mb, g.b, (uint64_t)g.N, (uint64_t)g.K, kBoxB))
        return cudaErrorInvalidValue;
    if (p.tma_out && !make_out_map(&mc, g.c, (uint64_t)g.M, (uint64_t)g.N, sizeof(Out) == 4, 32))
        return cudaErrorInvalidValue;
    const size_t smem = (size_t)T::stages * T::bytes + kEpiWarps * kStageOut + 1024;
    const auto k = gemm_tile_kernel<BN, Out, S>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess)
        return e;
    p.stall = g_stall_product.load() ? (uint32_t)g_stall_product.exchange(0) : 0u;
    p.spin = p.stall ? kStalledSpin : kGemmSpin;
    const uint32_t tiles = p.mt * p.nt;
    p.cut = cut;
    p.whole = cut ? tiles - tiles % (uint32_t)sms : tiles;
    p.items = p.whole + ((tiles - p.whole) << cut);
    return launch_dependent<S>(k, dim3(S > 1 ? p.items * S : std::min(p.items, (uint32_t)sms)), kTileThreads, smem, s, ma,
                               mb, mc, p);
}

template <int NT, typename Out>
cudaError_t run_small(const GemmArgs &g, int sms, cudaStream_t s)
{
    const dim3 grid((unsigned)((g.N + 15) / 16), (unsigned)((g.M + 8 * NT - 1) / (8 * NT)));
    // More than one block of K a warp: twice the warps, where all CTAs are on the
    // SMs at once (16 x 2048 x 1280 2.4 against 2.7 us, 31 x 53 x 4224 6.4 against
    // 8.9; 16 x 8192 x 8192 23.5 against 17.6) or small (8 x 8192 x 8192 12.0 against
    // 12.8).
    if (g.K > 8 * 128 && (NT == 1 || grid.x * grid.y <= (unsigned)sms))
        return launch_dependent(gemm_small_kernel<NT, 16, Out>, grid, 512, 0, s, g.a, g.sa, g.b, g.sb, (uint32_t)g.M,
                                (uint32_t)g.N, (uint32_t)g.K, static_cast<Out *>(g.c));
    return launch_dependent(gemm_small_kernel<NT, 8, Out>, grid, 256, 0, s, g.a, g.sa, g.b, g.sb, (uint32_t)g.M,
                            (uint32_t)g.N, (uint32_t)g.K, static_cast<Out *>(g.c));
}

template <typename Out>
cudaError_t gemm(const GemmArgs &g, cudaStream_t s)
{
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return e;
    if (g.M <= kSmallM || (g.M <= kSmallMaxM && g.M * g.N <= kSmallWork / std::max<int64_t>(g.K, 1024))) {
        if (g.M <= 8)
            return run_small<1, Out>(g, sms, s);
        if (g.M <= 16)
            return run_small<2, Out>(g, sms, s);
        return run_small<4, Out>(g, sms, s);
    }
    // Tile width: the fewest rounds of tiles on the SMs, each at what a step of
    // that width took (0.57, 0.38 and 0.28 us).  A last round of few tiles of 256
    // columns is cut into halves or quarters of their columns.
    const double step[3] = {0.57, 0.38, 0.28};
    const int64_t mt = (g.M + 127) / 128, wide = mt * ((g.N + 255) / 256), last = wide % sms;
    const auto rounds = [&](int64_t items) { return (double)((items + sms - 1) / sms); };
    double best = rounds(wide) * step[0];
    int bn = 256;
    uint32_t cut = 0;
    for (uint32_t i = 1; i <= 2; ++i) {
        const double parts = rounds(wide - last) * step[0] + rounds(last << i) * step[i];
        const double all = rounds(mt * ((g.N + (256 >> i) - 1) / (256 >> i))) * step[i];
        if (wide > sms && parts < best) {
            best = parts;
            bn = 256;
            cut = i;
        }
        if (all < best) {
            best = all;
            bn = 256 >> i;
            cut = 0;
        }
    }
    // Few tiles: clusters of 2 or 4 CTAs share the steps of a tile,
    // at about 1.5 and 2.3 us for the join (64 x 2560 x 2048 6.6 us alone, 6.0 in
    // pairs; 64 x 1536 x 2048 6.9, 6.0 and 5.4; 64 x 512 x 8192 18.9, 12.0 and 8.3;
    // 64 x 2048 x 1280 5.0 and 5.3).  32 clusters of 4 are on the SMs at a time, 36
    // are not.
    const int64_t kb = (g.K + 127) / 128;
    best *= (double)kb;
    int share = 1;
    for (uint32_t i = 1; i <= 2; ++i) {
        const int64_t items = mt * ((g.N + (256 >> i) - 1) / (256 >> i));
        const double pairs = 1.5 + step[i] * (double)((kb + 1) / 2), fours = 2.3 + step[i] * (double)((kb + 3) / 4);
        if (items * 2 <= sms && pairs < best) {
            best = pairs;
            bn = 256 >> i;
            share = 2;
        }
        if (items <= 32 && fours < best) {
            best = fours;
            bn = 256 >> i;
            share = 4;
        }
    }
    if (share == 2)
        return bn == 128 ? run_tile<128, Out, 2>(g, sms, 0, s) : run_tile<64, Out, 2>(g, sms, 0, s);
    if (share == 4)
        return bn == 128 ? run_tile<128, Out, 4>(g, sms, 0, s) : run_tile<64, Out, 4>(g, sms, 0, s);
    if (bn == 256)
        return run_tile<256, Out, 1>(g, sms, cut, s);
    return bn == 128 ? run_tile<128, Out, 1>(g, sms, 0, s) : run_tile<64, Out, 1>(g, sms, 0, s);
}

} // namespace

cudaError_t launch_gemm_fp8(const GemmArgs &g, int out_f32, cudaStream_t s)
{
    return out_f32 ? gemm<float>(g, s) : gemm<__nv_bfloat16>(g, s);
}

} // namespace mxq

extern "C" MXQ_API void mxq_test_stall_next_product(int on)
{
    mxq::g_stall_product.store(on == 1 || on == 2 ? on : 0);
}
