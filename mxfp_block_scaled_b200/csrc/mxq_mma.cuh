// mxq_mma.cuh -- what the kernels that multiply quantized operands by mma.sync
// share (sm_100a): asynchronous copies into shared memory, decoders of codes and
// scales into mma operands, and 16-bit rows of activations.
#pragma once

#include "mxq_device.cuh"

namespace mxq {

__device__ __forceinline__ void cp16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_small(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t lds32(const char *p) { return *reinterpret_cast<const uint32_t *>(p); }
__device__ __forceinline__ uint2 lds64(const char *p) { return *reinterpret_cast<const uint2 *>(p); }
__device__ __forceinline__ uint4 lds128(const char *p) { return *reinterpret_cast<const uint4 *>(p); }

// 16 bytes (zeros where `ok` is 0) into shared memory.
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void *src, bool ok)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16u : 0u) : "memory");
}

// The same of data that is read once: what it displaces in the second-level cache first
// is its like, not the code and the small operands of the next kernels.
__device__ __forceinline__ uint64_t once_policy()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void cp16_once(uint32_t dst, const void *src, bool ok, uint64_t policy)
{
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;"
                 ::"r"(dst), "l"(src), "r"(ok ? 16u : 0u), "l"(policy) : "memory");
}

// c += A B: A 16 rows x 16 k (f16), B 16 k x 8 columns (f16).
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four UE8M0 bytes -> fp32 2^(b - 127) (255 is NaN), through bf16, which
// holds them all.
__device__ __forceinline__ void ue8m0x4(uint32_t w, float (&d)[4])
{
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.bf16x2.ue8m0x2 %0, l;\n\t"
        "cvt.rn.bf16x2.ue8m0x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
    d[0] = bf16_lo(lo);
    d[1] = bf16_hi(lo);
    d[2] = bf16_lo(hi);
    d[3] = bf16_hi(hi);
}

// The four bytes of `w` (eight E2M1 codes) -> four f16x2 values, exact; the
// bytes are named inside one asm so that no shift is spent on them (by
// e2m1x8_to_f16x2, with shifts, 16 MXFP4 tokens take 82.7 us for 72.4, 64 NVFP4 ones
// 240 for 228).  For words from memory only, see e2m1x2.
__device__ __forceinline__ void e2m1x8_unpack(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}

// Four E4M3 codes -> two f16x2, exact.
__device__ __forceinline__ void e4m3x4_unpack(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}

// The low half of an f16x2 in both halves (an operand selector, no instruction).
__device__ __forceinline__ uint32_t low2(uint32_t h)
{
    const __half2 r = __low2half2(*reinterpret_cast<const __half2 *>(&h));
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ uint32_t high2(uint32_t h)
{
    const __half2 r = __high2half2(*reinterpret_cast<const __half2 *>(&h));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// c = A B of the same.
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// Power of two that brings a magnitude of these fp32 bits into [2^14, 2^15),
// as the bits of its factor; 1 for zero, Inf and NaN.  The exponent is kept
// within 126, so tiny rows land lower.
__device__ __forceinline__ float row_factor(uint32_t amax_bits)
{
    const int e = (int)(amax_bits >> 23) - 127;
    if (amax_bits == 0u || e == 128)
        return 1.0f;
    return __uint_as_float((uint32_t)(127 + min(max(14 - e, -126), 126)) << 23);
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

} // namespace mxq
