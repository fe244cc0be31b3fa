// attention.cuh -- how the attention kernels divide their work (sm_100a).
//
// A tile is up to R rows (a new token and a query head each) of one sequence and
// key/value head: row r is new token r / group and head r % group of the group.  A
// step is a tile and 2^LOG keys from a multiple of 2^LOG on; a tile has those of
// the keys that its last row sees, and one at least.  All steps in a row, by
// sequence, head, tile and key, are divided evenly among the CTAs, whatever tile
// boundaries lie between: no CTA has more than another by more than one step, and
// each leaves at most two tiles unfinished, the one it begins with and the one it
// ends with.  Unfinished tiles are left in the workspace (`part`), and
// attention_join_kernel adds up the parts of each in the order of the keys: no
// atomics, and the division follows from the lengths, the sizes and the number of
// SMs alone.  Every warp works its CTA's range out for itself, in the same way (out of
// line: a launch begins with cold instruction caches, and inlined in every role the
// division was most of a kernel's code).  What is out of line takes the arguments from a
// copy in shared memory: by a reference to the kernel's own they come from global memory,
// cold and one after the other.
#pragma once

#include "mxq_cache.cuh"
#include "mxq.h"

namespace mxq {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// Weights are 2^(s - r), s a row's scores in powers of two.  The reference r is kTop below the
// row's maximum when it is taken, and stays until a score lies more than kLag above it: the largest
// weight is 2^kTop to 2^kLag, the top of f16's range, so that a weight keeps 11 bits down to 2^-21
// of the largest and some down to 2^-31.  (The range is one of long contexts: with a maximum of 1,
// 2^18 tokens whose weights are 2^-25 of a first token's lost all that they give.)
constexpr float kTop = 7.0f, kLag = 15.0f;
constexpr float kLowest = -3e38f;       // a reference before the first key

// What a CTA leaves of the tile that it begins and does not finish (parts 0: none).
struct Unfinished {
    uint32_t first;             // the sequence's first row
    uint32_t row0, rows;        // the tile's first row, and the sequence's rows
    uint32_t head;
    uint32_t parts;             // the CTAs from this one on that have a part
    uint32_t pad[3];
};

struct AttArgs {
    CacheView c;
    const uint16_t *q;
    int64_t q_stride;
    uint32_t T, group, max_new;
    uint32_t over, upto;        // the sequences of this launch: those of over < rows <= upto
    uint32_t min_steps;         // of a CTA, where there are few
    uint32_t extra;             // steps that stand for what a tile costs beside its keys, before its first
    uint32_t tiles;             // of a sequence and head, at most
    float scale;                // softmax scale times log2(e)
    uint16_t *o;
    float *lse;
    Unfinished *left;           // [CTA]
    float *part;                // [CTA][2][R][dim] outputs of its keys alone, [R][2] references and sums
    FastDiv groupdiv;
    uint32_t spin;              // tests of a barrier before a wait gives up (tiles)
    uint32_t stall;             // test hook: CTA 0 withholds 1 + 2 t: keys, 2 + 2 t: values of its step t
};

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 1 / x, off by a unit of the last place; 0 for a sum of no keys.
__device__ __forceinline__ float inverse(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return x == 0.0f ? 0.0f : r;
}

// MXFP8 values enter the products relative to a power of two, 2^(ref - 134) where `ref` is a
// scale byte: codes times 2^(their scale - ref + 7), in f16.  It follows the scales of the keys at
// hand, and the output so far is rescaled where it moves (fp32, exact): no power enters the weights or
// their sum, so a large value takes nothing from tokens that are multiplied apart from it.  What
// kZeros and below count as is left to it; and it stays within 2^60 of the largest so far, so that no
// output leaves fp32.
constexpr uint32_t kZeros = 27, kSpan = 60;
struct ValueRef {
    uint32_t ref = kZeros, most = kZeros;

    // For keys whose largest scale is `top`, which may lie `slack` below the reference: the factor of
    // the output so far.
    __device__ __forceinline__ float follow(uint32_t top, uint32_t slack)
    {
        if (top <= ref && (top + slack >= ref || top <= kZeros))
            return 1.0f;
        const float f = move(max(top, max(most, kSpan) - kSpan));
        most = max(most, ref);
        return f;
    }
    __device__ __forceinline__ float move(uint32_t to)
    {
        const float f = __uint_as_float((uint32_t)max(127 + (int)ref - (int)to, 0) << 23);
        ref = to;
        return f;
    }
    __device__ __forceinline__ float unit() const { return __uint_as_float((ref - 7u) << 23); }
};

// Sequence b as this launch sees it: rows 0 where it is another launch's, or invalid (one
// that is longer than its row of the table among them: the length bounds the work).
struct Sequence {
    uint32_t first, n, rows;
    int64_t len;
};
__device__ __forceinline__ Sequence sequence(const AttArgs &a, uint32_t b)
{
    Sequence s;
    s.n = new_tokens(a.c, b, a.T, s.first);
    s.len = max(__ldg(a.c.lens + b), 0);
    if (s.n > a.max_new || (s.n > 0u && s.len > (int64_t)a.c.width << a.c.page_log)) {
        atomicOr(a.c.status, MXQ_DEV_INVALID_PAGE);
        s.n = 0;
    }
    s.rows = s.n * a.group;
    if (s.rows <= a.over || s.rows > a.upto)
        s.n = s.rows = 0;
    return s;
}

template <uint32_t R, uint32_t LOG>
struct Division {
    // Keys that tile `rt` sees, and its steps.
    static __device__ __forceinline__ uint32_t keys(const AttArgs &a, const Sequence &s, uint32_t rt)
    {
        const uint32_t last = min((rt + 1u) * R, s.rows) - 1u;
        return (uint32_t)max(s.len - s.n + fastdiv(last, a.groupdiv) + 1, (int64_t)0);
    }
    static __device__ __forceinline__ uint32_t steps(const AttArgs &a, const Sequence &s, uint32_t rt)
    {
        return max((keys(a, s, rt) + (1u << LOG) - 1u) >> LOG, 1u) + a.extra;
    }
    static __device__ __forceinline__ uint32_t tiles(const Sequence &s) { return (s.rows + R - 1u) / R; }

    // Steps of a key/value head of sequence s, all lanes of the warp together.
    static __device__ __forceinline__ uint64_t head_steps(const AttArgs &a, const Sequence &s)
    {
        uint64_t v = 0;
        for (uint32_t rt = threadIdx.x & 31u; rt < tiles(s); rt += 32u)
            v += steps(a, s, rt);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        return v;
    }

    // A sequence a lane: steps of all heads of sequence b (0 past the last).
    static __device__ __noinline__ uint64_t lane_steps(const AttArgs &a, uint32_t b)
    {
        Sequence s = {};
        if (b < a.c.seqs)
            s = sequence(a, b);
        const uint32_t nt = tiles(s);
        uint64_t v = 0;
        if (nt <= 4u)
            for (uint32_t rt = 0; rt < nt; ++rt)
                v += steps(a, s, rt);
        for (uint32_t many = __ballot_sync(0xFFFFFFFFu, nt > 4u); many; many &= many - 1u) {
            const uint32_t lane = __ffs(many) - 1;
            Sequence w;
            w.first = 0;
            w.n = __shfl_sync(0xFFFFFFFFu, s.n, lane);
            w.rows = __shfl_sync(0xFFFFFFFFu, s.rows, lane);
            w.len = __shfl_sync(0xFFFFFFFFu, s.len, lane);
            const uint64_t u = head_steps(a, w);
            if ((threadIdx.x & 31u) == lane)
                v = u;
        }
        return v * a.c.heads;
    }
};

// Where a CTA's range of steps begins and ends; in shared memory.
struct Range {
    uint64_t sums[32];
    uint64_t begin, end;        // steps of this CTA
    uint64_t total;
    uint32_t ctas;              // that have steps
    uint32_t b;                 // sequence of the first step, and its place there
    uint64_t at;
};

// Sum of v over the CTA, the same in every thread; `before`: over the threads before this one.
__device__ __forceinline__ uint64_t block_sum(uint64_t v, Range &r, uint64_t &before)
{
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    uint64_t s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t u = __shfl_up_sync(0xFFFFFFFFu, s, o);
        s += lane >= (uint32_t)o ? u : 0ull;
    }
    __syncthreads();
    if (lane == 31u)
        r.sums[warp] = s;
    __syncthreads();
    uint64_t total = 0;
    before = s - v;
    for (uint32_t w = 0; w < blockDim.x >> 5; ++w) {
        before += w < warp ? r.sums[w] : 0ull;
        total += r.sums[w];
    }
    return total;
}

// All threads: this CTA's range.
template <typename Div>
__device__ __noinline__ void find_range(const AttArgs &a, Range &r)
{
    uint64_t own = 0, before, v = 0;
    for (uint32_t b0 = 0; b0 < a.c.seqs; b0 += blockDim.x)
        own += v = Div::lane_steps(a, b0 + threadIdx.x);
    const uint64_t total = block_sum(own, r, before);
    const uint32_t ctas = (uint32_t)max(min((uint64_t)gridDim.x, total / a.min_steps), (uint64_t)1);
    const uint64_t begin = blockIdx.x < ctas ? total * blockIdx.x / ctas : total;
    const uint64_t end = blockIdx.x < ctas ? total * (blockIdx.x + 1u) / ctas : total;
    if (threadIdx.x == 0) {
        r.begin = begin;
        r.end = end;
        r.total = total;
        r.ctas = ctas;
    }
    if (begin < end) {
        uint64_t base = 0;
        for (uint32_t b0 = 0; b0 < a.c.seqs && base <= begin; b0 += blockDim.x) {
            if (a.c.seqs > blockDim.x)
                v = Div::lane_steps(a, b0 + threadIdx.x);
            const uint64_t sum = block_sum(v, r, before);
            if (begin >= base + before && begin < base + before + v) {
                r.b = b0 + threadIdx.x;
                r.at = begin - base - before;
            }
            base += sum;
        }
    }
    __syncthreads();
}

// A warp's walk over the pieces of its CTA's range: a tile, or the part of it in
// the range, or MOST steps of that, one after the other.  The tensor cores cut their sums
// to fp32 rather than round them, 16 keys at a time, which adds up to 2^-24 of the sum each:
// pieces keep it below 2^-12 (in one piece outputs over 2^20 tokens came out 0.7 % small).
// It lies in shared memory; all lanes call.
template <uint32_t R, uint32_t LOG, uint32_t MOST>
struct Walk {
    using Div = Division<R, LOG>;
    uint64_t left;              // steps of the range after this piece
    Sequence s;
    uint32_t b, head, rt;
    uint32_t k0, k1, steps;     // the piece's steps of the tile's
    uint32_t begun;             // the CTA's first step of the tile
    uint32_t keys;              // the tile's keys

    // The CTA has the tile to itself, and this piece ends it; pieces of the same tile came before.
    __device__ __forceinline__ bool whole() const { return begun == 0u && k1 == steps; }
    __device__ __forceinline__ bool earlier() const { return k0 > begun; }
    // The first of two unfinished tiles of a CTA is the one it did not begin.
    __device__ __forceinline__ uint32_t slot() const { return begun == 0u; }
    __device__ __forceinline__ bool unfinished() const { return begun == 0u && k1 < steps && left == 0u; }
    // The piece's first step of keys, and the one behind its last.
    __device__ __forceinline__ uint32_t from(const AttArgs &a) const { return max(k0, a.extra) - a.extra; }
    __device__ __forceinline__ uint32_t to(const AttArgs &a) const { return max(k1, a.extra) - a.extra; }

    // The piece at the walk's place, of as many steps as the range has left; back to `out`.
    __device__ __forceinline__ void take(const AttArgs &a, Walk &out)
    {
        steps = Div::steps(a, s, rt);
        keys = Div::keys(a, s, rt);
        k1 = (uint32_t)min((uint64_t)min(steps, k0 + MOST), k0 + left);
        left -= k1 - k0;
        __syncwarp();
        if ((threadIdx.x & 31u) == 0u)
            out = *this;
        __syncwarp();
    }
    static __device__ __noinline__ bool begin(Walk &out, const AttArgs &a, const Range &r)
    {
        Walk w;
        w.left = r.end - r.begin;
        if (w.left == 0)
            return false;
        w.b = r.b;
        w.s = sequence(a, w.b);
        const uint64_t per = Div::head_steps(a, w.s);
        w.head = (uint32_t)(r.at / per);
        uint64_t at = r.at - w.head * per;
        // the tile: 32 at a time
        const uint32_t lane = threadIdx.x & 31u, nt = Div::tiles(w.s);
#pragma unroll 1
        for (w.rt = 0;; w.rt += 32u) {
            uint64_t v = w.rt + lane < nt ? Div::steps(a, w.s, w.rt + lane) : 0u;
            const uint64_t own = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
                v += lane >= (uint32_t)o ? u : 0ull;
            }
            const uint32_t past = __ballot_sync(0xFFFFFFFFu, v > at);
            if (past) {
                const uint32_t l = __ffs(past) - 1;
                at -= __shfl_sync(0xFFFFFFFFu, v - own, l);
                w.rt += l;
                break;
            }
            at -= __shfl_sync(0xFFFFFFFFu, v, 31);
            if (w.rt + 32u >= nt)       // cannot be: the range lies in the sequence
                return false;
        }
        w.k0 = w.begun = (uint32_t)at;
        w.take(a, out);
        return true;
    }
    static __device__ __noinline__ bool next(Walk &out, const AttArgs &a)
    {
        Walk w = out;
        if (w.left == 0)
            return false;
        if (w.k1 < w.steps) {
            w.k0 = w.k1;
            w.take(a, out);
            return true;
        }
        w.k0 = w.begun = 0;
        if (++w.rt == Div::tiles(w.s)) {
            w.rt = 0;
            if (++w.head == a.c.heads) {
                w.head = 0;
                do {
                    if (++w.b >= a.c.seqs)
                        return false;
                    w.s = sequence(a, w.b);
                } while (w.s.rows == 0);
            }
        }
        w.take(a, out);
        return true;
    }
};

// CTAs from this one on that have a part of the tile that the range's last piece
// (of k steps so far) begins.
__device__ __forceinline__ uint32_t parts_of(const Range &r, uint32_t steps, uint32_t done)
{
    const uint64_t last = r.end - done + steps - 1u;            // the tile's last step
    // the CTA of a step x: the largest c with total c / ctas <= x
    return (uint32_t)(((last + 1u) * r.ctas + r.total - 1u) / r.total) - blockIdx.x;
}

template <uint32_t R, int D>
__device__ __forceinline__ float *part_of(const AttArgs &a, uint32_t cta, uint32_t second)
{
    return a.part + (uint64_t)(cta * 2u + second) * (R * (D + 2));
}

} // namespace mxq
