// ea_cache.cuh - the device view of a KV cache (ea_cache in ea.h) and the
// arithmetic of its 8-bit blocks, shared by the kernels that read and write it.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "ea_device.cuh"

namespace ea {

struct CacheDev {
    void *code[2];          // K, V
    float *scale[2];
    int64_t s_outer, s_row, s_head;   // elements
    const int32_t *table;   // nullptr: contiguous
    int64_t bt_stride;
    int rows, outer, cap, Hkv;
    int nsb;                // scale blocks of one (outer, head)
    int log2sb;
    int format;
};

// Checks a cache of B sequences and makes its device view; false: `why` says
// what is wrong with it.
bool cache_dev(const ea_cache *c, int B, CacheDev &d, ea_status &why);

// Row p of sequence b: the cache's outer index and row in it; false (reported)
// if its page is outside the cache.
__device__ __forceinline__ bool locate(const CacheDev &c, int b, int p, int &outer, int &row,
                                       uint32_t *err)
{
    if (!c.table) {
        outer = b;
        row = p;
        return true;
    }
    const int pg = p / c.rows;
    row = p - pg * c.rows;
    outer = c.table[b * c.bt_stride + pg];
    if (outer >= 0 && outer < c.outer)
        return true;
    raise_error(err, EA_DEVERR_CHECK);
    outer = 0;
    return false;
}

// Eight bf16 as floats.
__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint32_t amax8(const float (&x)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    return m;
}

// The scale of a block whose largest |value| has the float bits `amax`: the
// least 2^e, e >= -64, with amax <= qmax * 2^e.  With amax = 2^k * (1 + f):
// e4m3's qmax 448 = 2^8 * 1.75 and int8's 127 = 2^6 * 1.984375, so e is k - 8
// (k - 6) while 1 + f stays within that factor and one more above it.  NaN for
// an infinity or a NaN.
__device__ __forceinline__ float block_scale(uint32_t amax, bool e4m3)
{
    if (amax >= 0x7f800000u)
        return __uint_as_float(0x7fc00000u);
    const int k = static_cast<int>(amax >> 23) - 127;
    const uint32_t f = amax & 0x7fffffu;
    int e = e4m3 ? k - 8 + (f > 0x600000u ? 1 : 0) : k - 6 + (f > 0x7e0000u ? 1 : 0);
    e = e < -64 ? -64 : e;
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Four codes of values already divided by the scale, packed.  int8: adding
// 1.5 * 2^23 leaves the value, rounded to an integer (ties to even), in the low
// byte.
template <bool E4M3>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d)
{
    if constexpr (E4M3) {
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
        return static_cast<uint32_t>(lo) | static_cast<uint32_t>(hi) << 16;
    } else {
        const float M = 12582912.f;
        const uint32_t lo = __byte_perm(__float_as_uint(__fadd_rn(a, M)), __float_as_uint(__fadd_rn(b, M)), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(__fadd_rn(c, M)), __float_as_uint(__fadd_rn(d, M)), 0x0040);
        return __byte_perm(lo, hi, 0x5410);
    }
}

// The numbers that four packed codes stand for (before the scale), exact in f16:
// codes (0, 1) and (2, 3), or, paired the other way, (0, 2) and (1, 3).  int8:
// c + 128 placed in the fraction of 1024, minus 1152.
template <bool E4M3, bool APART = false>
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    if constexpr (E4M3) {
        if constexpr (APART)
            w = __byte_perm(w, 0u, 0x3120);
        asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t a = __byte_perm(u, 0x64646464u, APART ? 0x4240 : 0x4140);
        const uint32_t b = __byte_perm(u, 0x64646464u, APART ? 0x4341 : 0x4342);
        const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
        const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), off);
        const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&b), off);
        lo = *reinterpret_cast<const uint32_t *>(&x);
        hi = *reinterpret_cast<const uint32_t *>(&y);
    }
}

// Four codes of f16 numbers (codes times a power of two f).  Rounded once: the
// product is exact in f16 wherever it does not round to the code 0, and int8's
// sum with 1536 is fused with it.
template <bool E4M3>
__device__ __forceinline__ uint32_t encode4_f16(uint32_t lo, uint32_t hi, __half2 f)
{
    const __half2 a = *reinterpret_cast<const __half2 *>(&lo), b = *reinterpret_cast<const __half2 *>(&hi);
    if constexpr (E4M3) {
        const __half2 x = __hmul2(a, f), y = __hmul2(b, f);
        uint16_t p, q;
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(p) : "r"(*reinterpret_cast<const uint32_t *>(&x)));
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(q) : "r"(*reinterpret_cast<const uint32_t *>(&y)));
        return static_cast<uint32_t>(p) | static_cast<uint32_t>(q) << 16;
    } else {
        const __half2 m = __halves2half2(__ushort_as_half(0x6600), __ushort_as_half(0x6600));
        const __half2 x = __hfma2(a, f, m), y = __hfma2(b, f, m);
        return __byte_perm(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y), 0x6420);
    }
}

__device__ __forceinline__ float2 f16_f32(uint32_t h)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

} // namespace ea
