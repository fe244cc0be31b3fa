// mxq_cache.cuh -- where the tokens of a paged cache lie (sm_100a).
//
// A batch of sequences: cu[b] .. cu[b + 1] are the rows of sequence b's new
// tokens, lens[b] the tokens it has in the cache, those among them, and
// table[b, i] the page that holds its tokens i 2^page_log and on.  All of it
// is device data and nothing of it is trusted: every index is compared with
// its bound before it is used.
#pragma once

#include "mxq_device.cuh"
#include "mxq_layer.h"

namespace mxq {

// Number of the sequence that row `row` belongs to (cu ascends; of any other the
// result is some number below seqs, or seqs).  All lanes of a warp call, with rows of
// their own that do not descend.  The warp looks for the first lane's row together, 32
// places of cu at a time, since a bisection is a chain of as many loads as log2(seqs);
// rows of sequences further on are looked for by bisection, from there.
__device__ __forceinline__ uint32_t find_sequence(const CacheView &c, uint32_t row)
{
    const uint32_t lane = threadIdx.x & 31u;
    const int64_t want = __shfl_sync(0xFFFFFFFFu, row, 0);
    uint32_t lo = 0, n = c.seqs;        // the last b with cu[b] <= want is in [lo, lo + n)
    while (n > 1u) {
        const uint32_t step = (n + 31u) / 32u, at = lo + lane * step;
        const bool below = lane * step < n && __ldg(c.cu + at) <= want;
        const uint32_t k = __popc(__ballot_sync(0xFFFFFFFFu, below));
        const uint32_t skip = k ? (k - 1u) * step : 0u;
        lo += skip;
        n = min(step, n - skip);
    }
    uint32_t hi = c.seqs;
    if (__ldg(c.cu + lo + 1) <= (int64_t)row)
        while (hi - lo > 1u) {
            const uint32_t mid = (lo + hi) >> 1;
            if (__ldg(c.cu + mid) <= (int64_t)row)
                lo = mid;
            else
                hi = mid;
        }
    return __ldg(c.cu + lo) <= (int64_t)row && (int64_t)row < __ldg(c.cu + lo + 1) ? lo : c.seqs;
}

// Rows r0 .. r1 - 1 are rows of the call, which has T.
__device__ __forceinline__ bool rows_ok(int32_t r0, int32_t r1, uint32_t T)
{
    return r0 >= 0 && r1 >= r0 && (uint32_t)r1 <= T;
}

// New tokens of sequence b; none, and the status bit, where cu descends or leaves the call's rows.
__device__ __forceinline__ uint32_t new_tokens(const CacheView &c, uint32_t b, uint32_t T, uint32_t &first)
{
    const int32_t r0 = __ldg(c.cu + b), r1 = __ldg(c.cu + b + 1);
    first = (uint32_t)r0;
    if (rows_ok(r0, r1, T))
        return (uint32_t)(r1 - r0);
    atomicOr(c.status, MXQ_DEV_INVALID_PAGE);
    return 0u;
}

// What the table says of position `pos` of sequence b: a page, or a number that is none
// (c.pages where the table ends before).
__device__ __forceinline__ uint32_t table_entry(const CacheView &c, uint32_t b, uint32_t pos)
{
    const uint32_t i = pos >> c.page_log;
    return i < c.width ? (uint32_t)__ldg(c.table + (uint64_t)b * c.width + i) : c.pages;
}

// Page of position `pos` (at least 0) of sequence b; c.pages where the table
// has none, and the status bit set.
__device__ __forceinline__ uint32_t find_page(const CacheView &c, uint32_t b, uint32_t pos)
{
    const uint32_t page = table_entry(c, b, pos);
    if (page < c.pages)
        return page;
    atomicOr(c.status, MXQ_DEV_INVALID_PAGE);
    return c.pages;
}

// Number of the (page, head, token) row of codes that holds row `row`'s token;
// false where the row has no place: behind the last sequence, before the
// sequence's first position, of a sequence that leaves the call's T rows, or on an
// invalid page.  All lanes of a warp call, as above.
__device__ __forceinline__ bool find_place(const CacheView &c, uint32_t row, uint32_t T, uint64_t &at)
{
    const uint32_t b = find_sequence(c, row);
    if (b == c.seqs)
        return false;
    const int32_t end = __ldg(c.cu + b + 1);
    const int64_t pos = (int64_t)__ldg(c.lens + b) - end + row;
    if (pos < 0 || !rows_ok(__ldg(c.cu + b), end, T))
        return false;
    const uint32_t page = find_page(c, b, (uint32_t)pos);
    at = (((uint64_t)page * c.heads) << c.page_log) + ((uint32_t)pos & ((1u << c.page_log) - 1u));
    return page < c.pages;
}

} // namespace mxq
