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

cudaError_t launch_attention_rows(const AttArgs &a, int fmt, int dim, uint32_t sms, uint32_t &ctas, cudaStream_t s);
cudaError_t launch_attention_tiles(const AttArgs &a, int fmt, int dim, uint32_t ctas, cudaStream_t s);

namespace {

// Sequences of up to this many rows are attention_rows.cu's.
constexpr uint32_t kFewRows = 64;
constexpr uint32_t kMaxSms = 160;           // the division uses no more (workspace)
constexpr uint32_t kFewCtas = 4 * kMaxSms;  // of attention_rows.cu
constexpr uint32_t kFewTile = 16, kTile = 256;

size_t left_bytes() { return kFewCtas * sizeof(Unfinished); }
size_t rows_part_bytes(int64_t dim) { return (size_t)kFewCtas * 2 * kFewTile * (size_t)(dim + 2) * 4; }
size_t tiles_part_bytes(int64_t dim) { return (size_t)kMaxSms * 2 * (dim == 256 ? 128 : kTile) * (size_t)(dim + 2) * 4; }
bool few(int64_t group, int64_t max_new) { return group * max_new <= (int64_t)kFewRows; }

} // namespace

// The parts of a tile that CTA blockIdx.x of the kernel before began, added up in
// their order.  A warp takes a row, lanes its columns.
template <uint32_t R, int D>
__global__ void __launch_bounds__(256) attention_join_kernel(const AttArgs a)
{
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();
    const uint32_t lane = threadIdx.x & 31u, cta = blockIdx.x;
    const Unfinished u = a.left[cta];
    const uint32_t end = min(u.rows - u.row0, R);
    for (uint32_t r = blockIdx.y * 8u + (threadIdx.x >> 5); u.parts > 0u && r < end; r += gridDim.y * 8u) {
        // maximum over the parts: the first is the CTA's second, the others their CTAs' first
        float m = kLowest;
        for (uint32_t i = lane; i < u.parts; i += 32u)
            m = fmaxf(m, part_of<R, D>(a, cta + i, i == 0u)[R * D + r * 2u]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        constexpr int per = D / 32;
        float v[per], l = 0.0f;
#pragma unroll
        for (int j = 0; j < per; ++j)
            v[j] = 0.0f;
#pragma unroll 4
        for (uint32_t i = 0; i < u.parts; ++i) {
            const float *p = part_of<R, D>(a, cta + i, i == 0u);
            const float2 st = *reinterpret_cast<const float2 *>(p + R * D + r * 2u);
            const float f = ex2(st.x - m);
            l = fmaf(st.y, f, l);
#pragma unroll
            for (int j = 0; j < per; ++j)
                v[j] = fmaf(p[r * D + j * 32 + lane], f, v[j]);
        }
        const uint32_t row = u.row0 + r, i = fastdiv(row, a.groupdiv), h = u.head * a.group + row - i * a.group;
        const uint64_t out = (uint64_t)(u.first + i) * (a.c.heads * a.group) + h;
        const float f = l == 0.0f ? 0.0f : (a.c.v_s2 ? __ldg(a.c.v_s2 + u.head) : 1.0f) / l;
#pragma unroll
        for (int j = 0; j < per; ++j)
            reinterpret_cast<__nv_bfloat16 *>(a.o)[out * D + j * 32 + lane] = __float2bfloat16_rn(v[j] * f);
        if (lane == 0 && a.lse)
            a.lse[out] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
}

namespace {

template <uint32_t R>
cudaError_t join(const AttArgs &a, int dim, uint32_t ctas, cudaStream_t s)
{
    const dim3 grid(ctas, R == 16 ? 2 : 8);
    return dim == 64    ? launch_dependent(attention_join_kernel<R, 64>, grid, 256, 0, s, a)
           : dim == 128 ? launch_dependent(attention_join_kernel<R, 128>, grid, 256, 0, s, a)
                        : launch_dependent(attention_join_kernel<R == 256 ? 128 : R, 256>, grid, 256, 0, s, a);
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
    const uint32_t ctas = std::min<uint32_t>((uint32_t)sms, kMaxSms);
    const bool many = !few(a.group, c.max_new);
    // A lone sequence is one kernel's, whatever it has.
    const bool rows = !many || c.c.seqs > 1u;
    if (many) {
        a.over = rows ? kFewRows : 0u;
        a.upto = 0xFFFFFFFFu;
        a.min_steps = 4;
        e = launch_attention_tiles(a, fmt, dim, ctas, s);
        if (e == cudaSuccess)
            e = join<kTile>(a, dim, ctas, s);
    }
    if (rows && e == cudaSuccess) {
        a.over = 0;
        a.upto = many ? kFewRows : 0xFFFFFFFFu;
        a.min_steps = 8;
        uint32_t n = 0;         // at most kFewCtas
        e = launch_attention_rows(a, fmt, dim, ctas, n, s);
        if (e == cudaSuccess)
            e = join<kFewTile>(a, dim, n, s);
    }
    return e;
}

} // namespace mxq
