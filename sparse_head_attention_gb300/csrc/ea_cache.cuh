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

// Four codes of values already divided by the scale, packed.
template <bool E4M3>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d)
{
    if constexpr (E4M3) {
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
        return static_cast<uint32_t>(lo) | static_cast<uint32_t>(hi) << 16;
    } else {
        const int x = __float2int_rn(a), y = __float2int_rn(b), z = __float2int_rn(c),
                  w = __float2int_rn(d);
        return (x & 0xff) | (y & 0xff) << 8 | (z & 0xff) << 16 | static_cast<uint32_t>(w) << 24;
    }
}

// The numbers that four packed codes stand for (before the scale).
template <bool E4M3>
__device__ __forceinline__ void decode4(uint32_t w, float (&x)[4])
{
    if constexpr (E4M3) {
        uint32_t lo, hi;
        asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
        const float2 p = __half22float2(*reinterpret_cast<__half2 *>(&lo));
        const float2 q = __half22float2(*reinterpret_cast<__half2 *>(&hi));
        x[0] = p.x;
        x[1] = p.y;
        x[2] = q.x;
        x[3] = q.y;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
    }
}

} // namespace ea
