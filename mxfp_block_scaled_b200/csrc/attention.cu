// attention.cu -- attention of new tokens over a paged, quantized cache: which
// kernel takes which sequences, and the join of unfinished tiles (sm_100a).
//
//   s[j] = scale q . k_j (j <= the row's position),  p = softmax(s),
//   o = sum_j p_j v_j,  lse = ln sum_j exp(s[j]),
//
// for every row (a new token and a query head); the heads of a group share a
// key/value head.  k_j and v_j are the cache's codes times their block scales.
#include "attention.cuh"
#include <algorithm>

namespace mxq {

cudaError_t launch_attention_rows(const AttArgs &a, int fmt, int dim, uint32_t rows, uint32_t sms, uint64_t most_keys,
                                  uint32_t &ctas, cudaStream_t s);
cudaError_t launch_attention_tiles(const AttArgs &a, int fmt, int dim, uint32_t ctas, cudaStream_t s);

namespace {

// Sequences of up to kSomeRows rows are attention_rows.cu's; of MXFP8, where there are many
// keys, up to kFewRows: its 16 rows a tile decode a key again for every tile, while
// attention_tiles.cu takes 30 us to begin.  Measured, rows against tiles, 2 key/value heads.
// 64 sequences of up to 4096 with 32 rows: MXFP8 40 against 53 us (heads of 128), 72 against
// 89 (256); NVFP4 37 against 51, 52 against 71.  With 64 rows: MXFP8 59 against 58, 129
// against 100 (16 of 16384: 47 against 48, 85 against 69); NVFP4 53 against 54, 82 against
// 79.  8 of up to 500 with 64 rows (8192 keys times heads) 10 against 32, one of 30000
// (61440) 36 against 32.
constexpr uint32_t kFewRows = 32, kSomeRows = 64;
constexpr uint64_t kFewKeys = 1u << 16;     // times heads, as the table's width bounds them
constexpr uint32_t kMaxSms = 160;           // the division uses no more (workspace)
constexpr uint32_t kFewCtas = 5 * kMaxSms;  // of attention_rows.cu: 5 an SM with tiles of 8 rows, 4 with
constexpr uint32_t kFewTile = 16, kTile = 256;      // tiles of 16, whose parts are then the larger

size_t left_bytes() { return kFewCtas * sizeof(Unfinished); }
size_t rows_part_bytes(int64_t dim) { return (size_t)(4 * kMaxSms) * 2 * kFewTile * (size_t)(dim + 2) * 4; }
size_t tiles_part_bytes(int64_t dim) { return (size_t)kMaxSms * 2 * (dim == 256 ? 128 : kTile) * (size_t)(dim + 2) * 4; }
bool few(int64_t group, int64_t max_new) { return group * max_new <= (int64_t)kFewRows; }

} // namespace

// Parts of unfinished tiles, each its own keys' output, weighed by their sums and added up in
// their order.  Of the `ctas` CTAs of the kernel
// before, blockIdx.x counts those that began one; blockIdx.y its rows, 8 / WPR to a CTA.
// WPR warps share a row's parts, and their sums are added in the order of the warps;
// lanes have its columns.
template <uint32_t R, int D, uint32_t WPR>
__global__ void __launch_bounds__(256) attention_join_kernel(const __grid_constant__ AttArgs a, uint32_t ctas)
{
    __shared__ uint32_t found, count[8];
    __shared__ float sums[8][D];
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();
    if (tid == 0)
        found = ctas;
    uint32_t before = 0;
#pragma unroll 1
    for (uint32_t c0 = 0; c0 < ctas; c0 += 256u) {
        const bool has = c0 + tid < ctas && a.left[c0 + tid].parts > 0u;
        const uint32_t vote = __ballot_sync(0xFFFFFFFFu, has);
        __syncthreads();
        if (lane == 0)
            count[warp] = __popc(vote);
        __syncthreads();
        uint32_t at = before + __popc(vote & ((1u << lane) - 1u));
#pragma unroll
        for (uint32_t w = 0; w < 8u; ++w) {
            at += w < warp ? count[w] : 0u;
            before += count[w];
        }
        if (has && at == blockIdx.x)
            found = c0 + tid;
    }
    __syncthreads();
    const uint32_t cta = found;
    if (cta == ctas)
        return;
    const Unfinished u = a.left[cta];
    const uint32_t r = blockIdx.y * (8u / WPR) + warp / WPR, q = warp % WPR;
    const bool in = r < min(u.rows - u.row0, R);
    constexpr int per = D / 32;                 // neighbouring columns of a lane
    float v[per], l = 0.0f, m = kLowest;
#pragma unroll
    for (int j = 0; j < per; ++j)
        v[j] = 0.0f;
    if (in) {
        // maximum and sum over the parts: the first is the CTA's second, the others their CTAs' first
        auto stat = [&](uint32_t i) {
            return *reinterpret_cast<const float2 *>(part_of<R, D>(a, cta + i, i == 0u) + R * D + r * 2u);
        };
        const float2 own = lane < u.parts ? stat(lane) : make_float2(kLowest, 0.0f);
        m = own.x;
        for (uint32_t i = lane + 32u; i < u.parts; i += 32u)
            m = fmaxf(m, stat(i).x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        l = own.y * ex2(own.x - m);
        for (uint32_t i = lane + 32u; i < u.parts; i += 32u) {
            const float2 st = stat(i);
            l = fmaf(st.y, ex2(st.x - m), l);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
        const float inv = inverse(l);
#pragma unroll 8
        for (uint32_t i = q; i < u.parts; i += WPR) {
            const float *p = part_of<R, D>(a, cta + i, i == 0u);
            const float2 st = *reinterpret_cast<const float2 *>(p + R * D + r * 2u);
            float x[per];
            if constexpr (per == 2)
                *reinterpret_cast<float2 *>(x) = *reinterpret_cast<const float2 *>(p + r * D + lane * per);
            else
#pragma unroll
                for (int j = 0; j < per; j += 4)
                    *reinterpret_cast<float4 *>(x + j) = *reinterpret_cast<const float4 *>(p + r * D + lane * per + j);
            const float f = st.y * ex2(st.x - m) * inv;
#pragma unroll
            for (int j = 0; j < per; ++j)
                v[j] = fmaf(x[j], f, v[j]);
        }
    }
    if (WPR > 1u) {
#pragma unroll
        for (int j = 0; j < per; ++j)
            sums[warp][lane * per + j] = v[j];
        __syncthreads();
        if (q != 0u)
            return;
#pragma unroll
        for (uint32_t w = 1; w < WPR; ++w)
#pragma unroll
            for (int j = 0; j < per; ++j)
                v[j] += sums[warp + w][lane * per + j];
    }
    if (!in)
        return;
    const uint32_t row = u.row0 + r, i = fastdiv(row, a.groupdiv), h = u.head * a.group + row - i * a.group;
    const uint64_t out = (uint64_t)(u.first + i) * (a.c.heads * a.group) + h;
    const float f = a.c.v_s2 ? __ldg(a.c.v_s2 + u.head) : 1.0f;
#pragma unroll
    for (int j = 0; j < per; j += 2)
        *reinterpret_cast<__nv_bfloat162 *>(a.o + out * D + lane * per + j) = __floats2bfloat162_rn(v[j] * f, v[j + 1] * f);
    if (lane == 0 && a.lse)
        a.lse[out] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

namespace {

template <uint32_t R, int D>
cudaError_t join_of(const AttArgs &a, uint32_t ctas, uint32_t tiles, cudaStream_t s)
{
    // Few tiles have many parts: eight warps a row (a decoding step over 65536 tokens, 222
    // parts of each of two tiles, with one 50 us more; 64 sequences with 3 or 4 parts a tile
    // 1 us less with one).
    if (ctas > 8u * tiles)
        return launch_dependent(attention_join_kernel<R, D, 8>, dim3(tiles, R), 256, 0, s, a, ctas);
    return launch_dependent(attention_join_kernel<R, D, 1>, dim3(tiles, R / 8), 256, 0, s, a, ctas);
}

// Tiles there can be at most, and a CTA begins one unfinished at most.
template <uint32_t R>
cudaError_t join(const AttArgs &a, int dim, uint32_t ctas, cudaStream_t s)
{
    const uint32_t rows = dim == 256 && R == 256 ? 128 : R;
    const uint64_t tiles = a.c.heads * ((uint64_t)a.T * a.group / rows + a.c.seqs);
    const uint32_t n = (uint32_t)std::min<uint64_t>(tiles, ctas);
    return dim == 64    ? join_of<R, 64>(a, ctas, n, s)
           : dim == 128 ? join_of<R, 128>(a, ctas, n, s)
                        : join_of<R == 256 ? 128 : R, 256>(a, ctas, n, s);
}

} // namespace

// Both kernels' parts lie in the same place: one joins before the other begins.
size_t attention_workspace_bytes(int64_t group, int64_t head_dim, int64_t max_new)
{
    return left_bytes() + std::max(rows_part_bytes(head_dim), few(group, max_new) ? 0 : tiles_part_bytes(head_dim));
}

cudaError_t launch_attention(const AttentionCall &c, int fmt, int dim, cudaStream_t s)
{
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return e;
    AttArgs a;
    a.c = c.c;
    a.q = c.q;
    a.q_stride = c.q_stride;
    a.T = c.T;
    a.group = c.heads / c.c.heads;
    a.max_new = c.max_new;
    a.scale = c.scale * kLog2e;
    a.o = c.o;
    a.lse = c.lse;
    a.left = static_cast<Unfinished *>(c.workspace);
    a.part = reinterpret_cast<float *>(static_cast<char *>(c.workspace) + left_bytes());
    a.groupdiv = make_fastdiv(a.group);
    a.spin = a.stall = 0;       // the tiles' own
    const uint32_t ctas = std::min<uint32_t>((uint32_t)sms, kMaxSms);
    a.tiles = 0;
    const uint64_t keys = ((uint64_t)c.c.width << c.c.page_log) * c.c.seqs * c.c.heads;
    const uint32_t few_rows = fmt == MXQ_FMT_NVFP4 || keys <= kFewKeys ? kSomeRows : kFewRows;
    const bool many = (uint64_t)a.group * c.max_new > few_rows;
    // A lone sequence is one kernel's, whatever it has.
    const bool rows = !many || c.c.seqs > 1u;
    if (many) {
        a.over = rows ? few_rows : 0u;
        a.upto = 0xFFFFFFFFu;
        a.min_steps = 4;
        a.extra = 0;
        e = launch_attention_tiles(a, fmt, dim, ctas, s);
        if (e == cudaSuccess)
            e = join<kTile>(a, dim, ctas, s);
    }
    if (rows && e == cudaSuccess) {
        a.over = 0;
        a.upto = many ? few_rows : 0xFFFFFFFFu;
        a.min_steps = 8;
        // tiles of 8 rows where no sequence has more, else of 16
        const uint32_t most = std::max(many ? few_rows : a.max_new * a.group, 1u), rows_of = most <= 8u ? 8u : kFewTile;
        a.tiles = (most + rows_of - 1) / rows_of;
        // A tile's start costs a CTA about as much as 8 steps (its queries, the first copies,
        // the join of its warps).  Measured without and with: 64 sequences of up to 32768 69.3 and
        // 66.6 us, 64 of up to 4096 with 32 rows of 256 90 and 72; one sequence of 65536, with
        // few tiles to the CTAs, 28.2 and 28.2.
        a.extra = (uint64_t)c.c.seqs * c.c.heads * a.tiles * 16u >= ctas ? 8u : 0u;
        uint32_t n = 0;         // at most kFewCtas
        e = launch_attention_rows(a, fmt, dim, rows_of, ctas, (uint64_t)c.c.width << c.c.page_log, n, s);
        if (e == cudaSuccess && n > 0u)
            e = rows_of == 8u ? join<8>(a, dim, n, s) : join<kFewTile>(a, dim, n, s);
    }
    return e;
}

} // namespace mxq
