// ea_cache.cu - writing a KV cache (quantising to 8 bits with one scale per
// block of tokens and KV head), choosing the tokens that stay when it is cut by
// accumulated attention weight, and gathering those into another cache.
//
// All three only move data, so what bounds them is HBM for long inputs and the
// latency of a launch and a few dependent loads for short ones.
//   cache_write_kernel    one CTA per (block of tokens, KV head, sequence, K or
//                         V).  A row of a head is 16 threads x 16 bytes, so 128
//                         threads hold a whole block in registers: one read
//                         finds the block's largest value, sets the scale, and
//                         the same registers are rounded and stored.
//   cache_compact_kernel  the same over gathered rows of another cache, K's and
//                         V's block by one CTA (an index, a page and a row's
//                         place serve both).  From 8 bits to 8 bits it is the
//                         instructions that count: codes stay in f16 pairs (a
//                         power of two per row is exact there), ten or so for
//                         four codes instead of 50 in fp32.
//   evict_select_kernel   a cluster of CTAs per (sequence, KV head): the weights
//                         are read once into shared memory as ordered keys; a
//                         radix search (three digits, histograms summed over
//                         the cluster) finds the lightest that stays, and one
//                         ordered pass lists the tokens.  Bound by latency: a
//                         load, three cluster barriers, a few scans.
#include <cuda_runtime.h>

#include "ea_cache.cuh"
#include "ea_internal.h"

namespace ea {

constexpr int kCacheThreads = 128;
constexpr int kRowThreads = 16;                            // threads of one row: 8 elements each
constexpr int kRowsPerPass = kCacheThreads / kRowThreads;  // 8

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

// Maximum over the CTA (128 threads).
__device__ __forceinline__ uint32_t cta_max(uint32_t v, uint32_t *red)
{
    v = __reduce_max_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x / 32] = v;
    __syncthreads();
    return max(max(red[0], red[1]), max(red[2], red[3]));
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

struct WriteArgs {
    CacheDev c;
    const __nv_bfloat16 *x[2];
    int64_t n_sb, n_st, n_sh;
    const int32_t *start, *n_new;
    uint32_t *err;
    int T;
};

// Bound by HBM: 32K tokens of 8 heads into e4m3, 201 MB in 32.5 us (6.2 TB/s, 0.91
// of the measured copy rate).  One token each of 32 sequences, into blocks begun
// before, takes 3.1 us: the launch and three dependent loads.
template <int SB, int FMT>
__global__ void __launch_bounds__(kCacheThreads) cache_write_kernel(const WriteArgs a)
{
    constexpr bool kE4M3 = FMT == EA_CACHE_E4M3;
    constexpr int kPasses = SB / kRowsPerPass;
    __shared__ uint32_t red[4];
    const int h = blockIdx.x % a.c.Hkv, blk = blockIdx.x / a.c.Hkv;
    const int b = blockIdx.y, kv = blockIdx.z;
    const int start = a.start ? a.start[b] : 0, n = a.n_new ? a.n_new[b] : a.T;
    if (start < 0 || n < 0 || n > a.T || static_cast<int64_t>(start) + n > a.c.cap) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && kv == 0)
            raise_error(a.err, EA_DEVERR_CHECK);
        return;
    }
    const int p0 = (start / SB + blk) * SB;              // the block's first row
    const int lo = max(start, p0), hi = min(start + n, p0 + SB);
    if (lo >= hi)
        return;
    int outer, row0;
    if (!locate(a.c, b, p0, outer, row0, a.err))
        return;
    const int r = threadIdx.x / kRowThreads, e0 = threadIdx.x % kRowThreads * 8;
    const __nv_bfloat16 *src = a.x[kv] + b * a.n_sb + h * a.n_sh + e0;
    const int64_t dst0 = outer * a.c.s_outer + row0 * a.c.s_row + h * a.c.s_head + e0;

    uint4 raw[kPasses];
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int p = p0 + i * kRowsPerPass + r;
        raw[i] = make_uint4(0, 0, 0, 0);
        if (p >= lo && p < hi)
            raw[i] = __ldg(reinterpret_cast<const uint4 *>(src + (p - start) * a.n_st));
    }
    if constexpr (FMT == EA_CACHE_BF16) {
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.c.code[kv]) + dst0;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int p = p0 + i * kRowsPerPass + r;
            if (p >= lo && p < hi)
                *reinterpret_cast<uint4 *>(dst + (p - p0) * a.c.s_row) = raw[i];
        }
    } else {
        float x[8];
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            unpack8(raw[i], x);
            mx = max(mx, amax8(x));
        }
        float s = block_scale(cta_max(mx, red), kE4M3);
        float *sp = a.c.scale[kv] + (static_cast<int64_t>(outer) * a.c.Hkv + h) * a.c.nsb + row0 / SB;
        uint8_t *dst = static_cast<uint8_t *>(a.c.code[kv]) + dst0;
        if (lo > p0) {
            // the block already holds rows p0 .. lo - 1
            const float was = *sp;
            __syncthreads();                 // every thread has read it before it changes
            if (!(was <= s)) {
                s = isnan(s) ? s : was;      // larger, or NaN: it stays
            } else if (was < s) {
                const __half2 f = __float2half2_rn(was / s);   // below 1
#pragma unroll
                for (int i = 0; i < kPasses; ++i) {
                    const int k = i * kRowsPerPass + r;
                    if (p0 + k < lo) {
                        uint2 *w = reinterpret_cast<uint2 *>(dst + k * a.c.s_row);
                        uint32_t c[4];
                        codes_f16<kE4M3>(w->x, c[0], c[1]);
                        codes_f16<kE4M3>(w->y, c[2], c[3]);
                        *w = make_uint2(encode4_f16<kE4M3>(c[0], c[1], f), encode4_f16<kE4M3>(c[2], c[3], f));
                    }
                }
            }
        }
        if (threadIdx.x == 0)
            *sp = s;
        const float inv = isnan(s) ? 0.f : 1.f / s;          // a power of two: exact
        const bool dead = isnan(s);
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int p = p0 + i * kRowsPerPass + r;
            if (p >= lo && p < hi) {
                unpack8(raw[i], x);
                uint2 w = make_uint2(0u, 0u);
                if (!dead)
                    w = make_uint2(encode4<kE4M3>(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                                   encode4<kE4M3>(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
                *reinterpret_cast<uint2 *>(dst + (p - p0) * a.c.s_row) = w;
            }
        }
    }
}

// ------------------------------------------------------------ compaction
struct CompactArgs {
    CacheDev src, dst;
    const int32_t *index, *counts;
    const float *w;
    float *w_out;
    uint32_t *err;
    int keep;
};

// A thread's 16 bytes of a row as stored: 8 bf16 or 16 codes.
template <int FMT>
constexpr int kElems = FMT == EA_CACHE_BF16 ? 8 : 16;

__device__ __forceinline__ uint32_t word(const uint4 &v, int i)
{
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Their largest magnitude as float bits, scale applied.
template <int FMT>
__device__ __forceinline__ uint32_t row_amax(const uint4 &raw, float s)
{
    if constexpr (FMT == EA_CACHE_BF16) {
        float x[8];
        unpack8(raw, x);
        return amax8(x);
    } else {
        // the codes as they are, two to a word in its halves' upper bytes: e4m3's are
        // ordered by magnitude once the sign is off, int8's have their extremes
        constexpr uint32_t kUpper = FMT == EA_CACHE_E4M3 ? 0x7f007f00u : 0xff00ff00u;
        uint32_t top = 0u, bottom = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t even = word(raw, i) & kUpper, odd = (word(raw, i) << 8) & kUpper;
            top = __vmaxs2(top, __vmaxs2(even, odd));
            if constexpr (FMT == EA_CACHE_INT8)
                bottom = __vmins2(bottom, __vmins2(even, odd));
        }
        float m;
        if constexpr (FMT == EA_CACHE_E4M3) {
            uint32_t lo, hi;
            codes_f16<true>(max(top >> 24, (top >> 8) & 0xffu), lo, hi);
            m = __half2float(__ushort_as_half(static_cast<uint16_t>(lo)));
        } else {
            const int t = static_cast<int>(top), u = static_cast<int>(bottom);
            m = static_cast<float>(max(max(t >> 24, (t << 16) >> 24), -min(u >> 24, (u << 16) >> 24)));
        }
        return __float_as_uint(m * s) & 0x7fffffffu;
    }
}

__device__ __forceinline__ uint32_t times512(uint32_t h)
{
    const __half2 x = __hmul2(*reinterpret_cast<const __half2 *>(&h), __float2half2_rn(512.f));
    return *reinterpret_cast<const uint32_t *>(&x);
}

// Stores them as codes of a block of scale 1 / inv (zeros for a NaN scale).
template <int SRC, bool E4M3>
__device__ __forceinline__ void put_codes(uint8_t *dst, const uint4 &raw, float s, float inv, bool dead)
{
    if constexpr (SRC == EA_CACHE_BF16) {
        float x[8];
        unpack8(raw, x);
        const uint2 w = make_uint2(encode4<E4M3>(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                                   encode4<E4M3>(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
        *reinterpret_cast<uint2 *>(dst) = dead ? make_uint2(0u, 0u) : w;
    } else {
        // a row of the block's own scale keeps its codes as they are (a block of a
        // NaN scale has no such row)
        if (E4M3 == (SRC == EA_CACHE_E4M3) && s * inv == 1.f) {
            *reinterpret_cast<uint4 *>(dst) = raw;
            return;
        }
        // The ratio of the scales.  The block's scale is set by its largest value, so no
        // code times the ratio is beyond qmax, and f16 holds every product.  Int8's codes
        // are 1 at least, and the ratio 2^8 at most; e4m3's go down to 2^-9, and the ratio
        // up to 2^17, more than f16 holds: it is then applied as 2^9 and the rest, both
        // exact.  What is capped is the ratio of a row of zeros.
        const float ratio = s * inv;
        const bool two = SRC == EA_CACHE_E4M3 && ratio > 512.f;
        const __half2 f = __float2half2_rn(fminf(two ? ratio * 0x1p-9f : ratio, 512.f));
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t lo, hi;
            codes_f16<SRC == EA_CACHE_E4M3>(word(raw, i), lo, hi);
            if (two) {
                lo = times512(lo);
                hi = times512(hi);
            }
            w[i] = dead ? 0u : encode4_f16<E4M3>(lo, hi, f);
        }
        *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Stores them as bf16.
template <int SRC>
__device__ __forceinline__ void put_bf16(__nv_bfloat16 *dst, const uint4 &raw, float s)
{
    if constexpr (SRC == EA_CACHE_BF16) {
        *reinterpret_cast<uint4 *>(dst) = raw;
    } else {
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t c[2];
            codes_f16<SRC == EA_CACHE_E4M3>(word(raw, i), c[0], c[1]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float2 v = f16_f32(c[k]);
                o[2 * i + k] = pack_bf16x2(v.x * s, v.y * s);
            }
        }
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(o[0], o[1], o[2], o[3]);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

// Three dependent loads deep (index, page, data) with little work behind them, so
// what counts is how many are in flight: the index is read before the count is
// known, K's and V's rows are read together (8 bits) or by a CTA each (bf16), and
// registers are kept low enough for many CTAs (16 per SM with blocks of 32: 31 us,
// ten: 34).  After that it is instructions (67 % of the issue slots taken):
// magnitudes are compared as codes, not as numbers (34 -> 31 us), and a row whose
// scale stays is copied (31 -> 30).
// Measured: 16 paged int8 caches, 4000 of up to 16384 tokens kept, blocks of 32,
// 30.6 us (119 MB, 3.9 TB/s; the floor at the measured HBM rate is 17.6); 8192 of 32K
// bf16 tokens to e4m3, 51 MB, 9.7 us out of L2 and 14.4 out of HBM (floor 7.5; K and
// V by one CTA 16.3).
template <int SB, int SRC, int DST>
__global__ void __launch_bounds__(kCacheThreads, SB > 64 ? 3 : SRC == EA_CACHE_BF16 ? 10 : SB == 64 ? 6 : 14)
    cache_compact_kernel(const CompactArgs a)
{
    constexpr bool kE4M3 = DST == EA_CACHE_E4M3;
    constexpr int kRowThreads = EA_HEAD_DIM / kElems<SRC>, kRowsPerPass = kCacheThreads / kRowThreads;
    constexpr int kPasses = SB / kRowsPerPass;         // 1 at least: 16 rows a pass
    // K and V at once, or, where that takes too many registers, by a CTA each
    constexpr int KV = SRC == EA_CACHE_BF16 ? 1 : 2;
    const int kv0 = KV == 1 ? blockIdx.z : 0;
    using Elem = typename std::conditional<SRC == EA_CACHE_BF16, uint16_t, uint8_t>::type;
    __shared__ uint32_t red[2][4];
    const int h = blockIdx.x % a.dst.Hkv, blk = blockIdx.x / a.dst.Hkv;
    const int b = blockIdx.y, p0 = blk * SB;
    const int r = threadIdx.x / kRowThreads, e0 = threadIdx.x % kRowThreads * kElems<SRC>;
    const int64_t unit = static_cast<int64_t>(b) * a.dst.Hkv + h;
    const int32_t *index = a.index + unit * a.keep;
    int at[kPasses], so[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int p = p0 + i * kRowsPerPass + r;
        at[i] = p < a.keep ? __ldg(index + p) : -1;
    }
    const int n = a.counts[b];
    if (n < 0 || n > a.keep) {
        if (threadIdx.x == 0 && blockIdx.x == 0)
            raise_error(a.err, EA_DEVERR_CHECK);
        return;
    }
    if (p0 >= n)
        return;
    int outer, row0;
    if (!locate(a.dst, b, p0, outer, row0, a.err))
        return;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int p = p0 + i * kRowsPerPass + r;
        if (p >= n) {
            at[i] = -1;
        } else {
            if (at[i] < 0 || at[i] >= a.src.cap) {
                raise_error(a.err, EA_DEVERR_CHECK);
                at[i] = -1;
            }
            if (a.w && e0 == 0 && kv0 == 0)
                a.w_out[unit * a.dst.cap + p] = at[i] >= 0 ? __ldg(a.w + unit * a.src.cap + at[i]) : 0.f;
        }
        so[i] = b;
        if (a.src.table && at[i] >= 0) {
            int row;
            if (!locate(a.src, b, at[i], so[i], row, a.err))
                row = -1;
            at[i] = row;
        }
    }
    const int64_t src0 = h * a.src.s_head + e0;
    const int64_t dst0 = outer * a.dst.s_outer + row0 * a.dst.s_row + h * a.dst.s_head + e0;
    uint4 raw[KV][kPasses];
    float sc[KV][kPasses];
    auto load = [&](int kv, uint4 (&rw)[kPasses], float (&s)[kPasses]) {
        const Elem *src = static_cast<const Elem *>(a.src.code[kv]) + src0;
        const float *ssrc = a.src.scale[kv];
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            rw[i] = make_uint4(0u, 0u, 0u, 0u);
            s[i] = 1.f;
            if (at[i] >= 0) {
                rw[i] = __ldg(reinterpret_cast<const uint4 *>(src + so[i] * a.src.s_outer + at[i] * a.src.s_row));
                if constexpr (SRC != EA_CACHE_BF16)
                    s[i] = __ldg(ssrc + (static_cast<int64_t>(so[i]) * a.src.Hkv + h) * a.src.nsb +
                                 (at[i] >> a.src.log2sb));
            }
        }
    };
    if constexpr (KV == 2) {
        load(0, raw[0], sc[0]);
        load(1, raw[1], sc[1]);
    }
#pragma unroll
    for (int j = 0; j < KV; ++j) {
        const int kv = KV == 1 ? kv0 : j;
        uint4 (&rw)[kPasses] = raw[j];
        float (&s_row)[kPasses] = sc[j];
        if constexpr (KV == 1)
            load(kv, rw, s_row);
        if constexpr (DST == EA_CACHE_BF16) {
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.dst.code[kv]) + dst0;
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int k = i * kRowsPerPass + r;
                if (p0 + k < n)
                    put_bf16<SRC>(dst + k * a.dst.s_row, rw[i], s_row[i]);
            }
        } else {
            uint32_t mx = 0;
#pragma unroll
            for (int i = 0; i < kPasses; ++i)
                mx = max(mx, row_amax<SRC>(rw[i], s_row[i]));
            mx = cta_max(mx, red[j]);
            // A code whose value was rounded up to 2^128 has a finite scale (a block with a
            // NaN scale gives a NaN here): the largest fp32 gives the scale that it needs.
            if (SRC != EA_CACHE_BF16 && mx == 0x7f800000u)
                mx = 0x7f7fffffu;
            const float s = block_scale(mx, kE4M3);
            if (threadIdx.x == 0)
                a.dst.scale[kv][(static_cast<int64_t>(outer) * a.dst.Hkv + h) * a.dst.nsb + row0 / SB] = s;
            const bool dead = isnan(s);
            const float inv = 1.f / s;                  // a power of two: exact
            uint8_t *dst = static_cast<uint8_t *>(a.dst.code[kv]) + dst0;
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int k = i * kRowsPerPass + r;
                if (p0 + k < n)
                    put_codes<SRC, kE4M3>(dst + k * a.dst.s_row, rw[i], s_row[i], inv, dead);
            }
        }
    }
}

// ------------------------------------------------------------ selection
constexpr int kSelThreads = 1024;
constexpr int kSelBits = 11;                 // digits: bits 31..21, 20..10, 9..0
constexpr int kSelBins = 1 << kSelBits;
constexpr int kSelMaxCluster = 8;
constexpr int kSelMaxKeys = 46 * 1024;       // keys a CTA holds in shared memory at most

struct SelectArgs {
    const float *w;
    const int32_t *seqlens;
    int32_t *index, *new_seqlens;
    uint32_t *err;
    int Hkv, Lmax, keep, sink, recent;
    int cap;                                 // keys a CTA holds in shared memory
};

struct SelSmem {
    uint32_t hist[3][kSelBins];
    uint32_t coarse[3][kSelBins / 8];        // sums of eight bins each
    uint32_t warp[32];
    uint32_t digit, above;                   // result of one radix step
    uint32_t before[3];                      // tokens above the step's digit in the CTAs before this one
    uint32_t equal_before;                   // tokens at the threshold there
    uint32_t keys[];                         // [sel_place(cap)]
};

// Where key i of a CTA lies: a word is left out after every sixteen, so that
// threads that read runs of consecutive keys meet different banks.
__host__ __device__ __forceinline__ int sel_place(int i) { return i + (i >> 4); }

// Order-preserving bits of a weight: larger weight, larger key; -0 equals +0;
// a NaN is below everything.
__device__ __forceinline__ uint32_t weight_key(float f)
{
    if (isnan(f))
        return 0u;
    const uint32_t u = f == 0.f ? 0u : __float_as_uint(f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t cl_addr)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cl_addr) : "memory");
    return v;
}

// Inclusive sum over the CTA (1024 threads); `total` is the whole sum.
__device__ __forceinline__ uint32_t cta_scan(uint32_t v, uint32_t *warp_sums, uint32_t &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o)
            x += y;
    }
    __syncthreads();                          // warp_sums of the previous call have been read
    if (lane == 31)
        warp_sums[warp] = x;
    __syncthreads();
    uint32_t s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o)
            s += y;
    }
    total = __shfl_sync(0xffffffffu, s, 31);
    const uint32_t before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
    return x + (warp > 0 ? before : 0u);
}

// Bound by latency, not by what it reads (4.5 MB at most below): 8 heads of one
// 128K sequence, 8192 kept, 19.7 us; 32 ragged sequences of up to 20001, 2048 kept,
// 23.4 us: one read of the weights, then, one after the other, three digits (each a
// histogram, a cluster barrier and two scans) and the list.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const SelectArgs a)
{
    extern __shared__ __align__(16) uint8_t smem_raw[];
    SelSmem &sm = *reinterpret_cast<SelSmem *>(smem_raw);
    const int tid = threadIdx.x;
    const int C = gridDim.x, rank = blockIdx.x;        // one cluster spans the x dimension
    const int unit = blockIdx.y + gridDim.y * blockIdx.z;
    const int b = unit / a.Hkv;
    int L = a.seqlens[b];
    if (L < 0 || L > a.Lmax) {
        if (tid == 0 && rank == 0)
            raise_error(a.err, EA_DEVERR_CHECK);
        L = 0;
    }
    const int n_keep = min(L, a.keep);
    int32_t *out = a.index + static_cast<int64_t>(unit) * a.keep;
    if (tid == 0 && rank == 0 && unit % a.Hkv == 0)
        a.new_seqlens[b] = n_keep;
    // entries behind the kept ones
    for (int i = n_keep + rank * kSelThreads + tid; i < a.keep; i += C * kSelThreads)
        out[i] = -1;
    if (L <= a.keep) {                                  // the same in every CTA of the cluster
        for (int i = rank * kSelThreads + tid; i < L; i += C * kSelThreads)
            out[i] = i;
        return;
    }
    for (int i = tid; i < 3 * kSelBins; i += kSelThreads)
        (&sm.hist[0][0])[i] = 0u;
    if (tid < 3)
        sm.before[tid] = 0u;
    if (tid == 3)
        sm.equal_before = 0u;
    __syncthreads();

    // this CTA's share of the middle tokens [sink, L - recent): lo + 0 .. lo + n - 1
    const float *w = a.w + static_cast<int64_t>(unit) * a.Lmax;
    const int m0 = a.sink, m1 = L - a.recent;
    const int len = (m1 - m0 + C - 1) / C;
    const int lo = min(m0 + rank * len, m1), n = min(lo + len, m1) - lo;
    const int held = min(n, a.cap);                     // the rest (very long sequences) is read again
    auto key_at = [&](int i) { return i < held ? sm.keys[sel_place(i)] : weight_key(__ldg(w + lo + i)); };
    const uint32_t zero = weight_key(0.f);
    uint32_t zeros = 0;
#pragma unroll 8
    for (int i = tid; i < n; i += kSelThreads) {
        const uint32_t k = weight_key(__ldg(w + lo + i));
        if (i < held)
            sm.keys[sel_place(i)] = k;
        // tokens that were never looked at are many: counted here, not one by one in their bin
        if (k == zero)
            ++zeros;
        else
            atomicAdd(&sm.hist[0][k >> 21], 1u);
    }
    zeros = __reduce_add_sync(0xffffffffu, zeros);
    if ((tid & 31) == 0 && zeros)
        atomicAdd(&sm.hist[0][zero >> 21], zeros);

    uint32_t want = a.keep - a.sink - a.recent;         // tokens of the middle that stay (< m1 - m0)
    uint32_t prefix = 0;                                // the threshold's digits found so far
#pragma unroll 1
    for (int step = 0; step < 3; ++step) {
        const int shift = step == 0 ? 21 : step == 1 ? 10 : 0;
        const uint32_t mask = step == 2 ? 0x3ffu : 0x7ffu;
        if (step > 0) {
            const int up = step == 1 ? 21 : 10;
            auto count = [&](uint32_t k) {
                if ((k >> up) == prefix)
                    atomicAdd(&sm.hist[step][(k >> shift) & mask], 1u);
            };
#pragma unroll 8
            for (int i = tid; i < held; i += kSelThreads)
                count(sm.keys[sel_place(i)]);
            for (int i = held + tid; i < n; i += kSelThreads)
                count(weight_key(__ldg(w + lo + i)));
        }
        // Sums over the cluster are of eight bins each first (reading all 2048 bins
        // of eight CTAs took 4200 cycles a step), then of the eight that hold the
        // want-th largest.
        __syncthreads();
        if (tid < kSelBins / 8) {
            const uint4 u = *reinterpret_cast<const uint4 *>(&sm.hist[step][8 * tid]);
            const uint4 v = *reinterpret_cast<const uint4 *>(&sm.hist[step][8 * tid + 4]);
            sm.coarse[step][tid] = u.x + u.y + u.z + u.w + v.x + v.y + v.z + v.w;
        }
        cluster_sync_all();
        if (tid < 256) {
            // thread t: the coarse bin 255 - t, over the cluster and over the CTAs before this one
            uint32_t c = 0, before = 0;
            const uint32_t bin = smem_u32(&sm.coarse[step][255 - tid]);
#pragma unroll
            for (int r = 0; r < kSelMaxCluster; ++r)
                if (r < C) {
                    const uint32_t v = ld_cluster_u32(mapa_shared(bin, r));
                    c += v;
                    before += r < rank ? v : 0u;
                }
            uint32_t x = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
                if ((tid & 31) >= o)
                    x += y;
            }
            if ((tid & 31) == 31)
                sm.warp[tid >> 5] = x;
            named_bar_sync(1, 256);
            uint32_t excl = x - c;
#pragma unroll
            for (int k = 0; k < 7; ++k)
                excl += k < tid >> 5 ? sm.warp[k] : 0u;
            if (want > excl && want <= excl + c) {
                sm.digit = 255 - tid;
                sm.above = excl;
            }
            named_bar_sync(1, 256);
            const int coarse = sm.digit;
            named_bar_sync(1, 256);                      // read before the fine one replaces it
            if (want > 0 && 255 - tid > coarse && before)
                atomicAdd(&sm.before[step], before);
            // the eight bins, by the first warp: lane l takes bin 7 - l % 8 of CTAs l / 8 and l / 8 + 4
            if (tid < 32 && want > 0) {
                uint32_t all = 0, bef = 0;
                const uint32_t fine = smem_u32(&sm.hist[step][8 * coarse + 7 - (tid & 7)]);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int r = (tid >> 3) + 4 * k;
                    if (r < C) {
                        const uint32_t v = ld_cluster_u32(mapa_shared(fine, r));
                        all += v;
                        bef += r < rank ? v : 0u;
                    }
                }
#pragma unroll
                for (int o = 8; o < 32; o <<= 1) {
                    all += __shfl_xor_sync(0xffffffffu, all, o);
                    bef += __shfl_xor_sync(0xffffffffu, bef, o);
                }
                // lane l < 8: bins from the top
                uint32_t up = all, bup = bef;
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, up, o);
                    const uint32_t z = __shfl_up_sync(0xffffffffu, bup, o);
                    if ((tid & 7) >= o) {
                        up += y;
                        bup += z;
                    }
                }
                const uint32_t excl8 = sm.above + up - all;
                __syncwarp();
                if (tid < 8 && want > excl8 && want <= excl8 + all) {
                    sm.digit = 8 * coarse + 7 - tid;
                    sm.above = excl8;
                    if (bup - bef)
                        atomicAdd(&sm.before[step], bup - bef);
                    if (step == 2)
                        sm.equal_before = bef;
                }
            }
        }
        __syncthreads();
        if (want == 0)
            break;                                       // the same in every CTA
        want -= sm.above;
        prefix = step == 0 ? sm.digit : prefix << (step == 2 ? 10 : 11) | sm.digit;
    }
    // tokens with a key above `prefix` stay, and the first `want` of those equal to it
    const bool none = a.keep == a.sink + a.recent;
    const uint32_t thr = none ? 0xffffffffu : prefix;    // no key reaches 0xffffffff
    // ordered list: each thread takes its run of consecutive tokens, up to 32 (one
    // scan for up to 32K tokens of a CTA)
    uint32_t equal = none ? 0u : sm.equal_before;
    uint32_t pos = a.sink + (none ? 0u : sm.before[0] + sm.before[1] + sm.before[2]) + min(equal, want);
    for (int i0 = 0; i0 < n; i0 += 32 * kSelThreads) {
        const int per = min(32, (n - i0 + kSelThreads - 1) / kSelThreads);
        const int f = min(i0 + tid * per, n), e = min(f + per, n);
        uint32_t hi = 0, eqs = 0;                        // bit j: token f + j above / at the threshold
#pragma unroll 8
        for (int j = 0; j < e - f; ++j) {
            const uint32_t k = key_at(f + j);
            hi |= (k > thr ? 1u : 0u) << j;
            eqs |= (k == thr ? 1u : 0u) << j;
        }
        uint32_t total;
        const uint32_t mine = __popc(hi) << 16 | __popc(eqs);
        const uint32_t before = cta_scan(mine, sm.warp, total) - mine;
        const uint32_t eq = equal + (before & 0xffffu);  // equal ones before this thread's
        uint32_t at = pos + (before >> 16) + (min(eq, want) - min(equal, want));
        // of this thread's equal ones the first want - eq stay
        uint32_t stay = hi, left = want > eq ? want - eq : 0u;
        while (left > 0 && eqs) {
            stay |= eqs & (0u - eqs);
            eqs &= eqs - 1;
            --left;
        }
        while (stay) {
            out[at++] = lo + f + __ffs(stay) - 1;
            stay &= stay - 1;
        }
        pos += (total >> 16) + (min(equal + (total & 0xffffu), want) - min(equal, want));
        equal += total & 0xffffu;
    }
    // the protected tokens on both sides
    for (int i = rank * kSelThreads + tid; i < a.sink; i += C * kSelThreads)
        out[i] = i;
    for (int i = rank * kSelThreads + tid; i < a.recent; i += C * kSelThreads)
        out[a.keep - a.recent + i] = m1 + i;
    cluster_sync_all();                                  // no CTA leaves while its histograms may be read
}

// ------------------------------------------------------------ launches
bool cache_dev(const ea_cache *c, int B, CacheDev &d, ea_status &why)
{
    why = EA_ERR_INVALID_ARG;
    if (!c || !c->K || !c->V || c->format < EA_CACHE_BF16 || c->format > EA_CACHE_INT8 || c->rows < 1 ||
        c->outer < 1 || c->Hkv < 1 || B < 1)
        return false;
    const bool wide = c->format == EA_CACHE_BF16;
    const int sb = wide ? 64 : c->scale_block;
    if (!wide && (!c->k_scale || !c->v_scale))
        return false;
    if (c->d != EA_HEAD_DIM || (sb != 16 && sb != 32 && sb != 64 && sb != 128) || B > 65535 ||
        c->Hkv > 65535) {
        why = EA_ERR_UNSUPPORTED;
        return false;
    }
    if (c->kv_str[3] != 1)
        return false;
    const int unit = wide ? 8 : 16;                     // elements of 16 bytes
    for (int k = 0; k < 3; ++k)
        if (c->kv_str[k] <= 0 || c->kv_str[k] % unit)
            return false;
    for (const void *p : {static_cast<const void *>(c->K), static_cast<const void *>(c->V)})
        if (reinterpret_cast<uintptr_t>(p) & 15u)
            return false;
    int64_t cap = c->rows;
    if (c->block_table) {
        if (c->max_pages < 1 || c->bt_stride < c->max_pages)
            return false;
        if (!wide && c->rows % sb) {
            why = EA_ERR_UNSUPPORTED;
            return false;
        }
        cap = static_cast<int64_t>(c->rows) * c->max_pages;
    } else if (c->outer != B) {
        return false;
    }
    if (cap > (int64_t(1) << 31) - 256) {               // row numbers are 32-bit
        why = EA_ERR_UNSUPPORTED;
        return false;
    }
    d.code[0] = c->K;
    d.code[1] = c->V;
    d.scale[0] = c->k_scale;
    d.scale[1] = c->v_scale;
    d.s_outer = c->kv_str[0];
    d.s_row = c->kv_str[1];
    d.s_head = c->kv_str[2];
    d.table = c->block_table;
    d.bt_stride = c->bt_stride;
    d.rows = c->rows;
    d.outer = c->outer;
    d.cap = static_cast<int>(cap);
    d.Hkv = c->Hkv;
    d.nsb = static_cast<int>(ceil_div(c->rows, sb));
    d.log2sb = sb == 16 ? 4 : sb == 32 ? 5 : sb == 64 ? 6 : 7;
    d.format = c->format;
    why = EA_OK;
    return true;
}

static bool ws_ok(const void *ws, size_t bytes)
{
    return ws && !(reinterpret_cast<uintptr_t>(ws) & 255u) && bytes >= sizeof(ea_ws_header);
}

template <int SB>
static void launch_write(const WriteArgs &a, dim3 grid, cudaStream_t st)
{
    if (a.c.format == EA_CACHE_E4M3)
        cache_write_kernel<SB, EA_CACHE_E4M3><<<grid, kCacheThreads, 0, st>>>(a);
    else
        cache_write_kernel<SB, EA_CACHE_INT8><<<grid, kCacheThreads, 0, st>>>(a);
}

template <int SB, int SRC>
static void launch_compact_src(const CompactArgs &a, dim3 grid, cudaStream_t st)
{
    if (a.dst.format == EA_CACHE_E4M3)
        cache_compact_kernel<SB, SRC, EA_CACHE_E4M3><<<grid, kCacheThreads, 0, st>>>(a);
    else if (a.dst.format == EA_CACHE_INT8)
        cache_compact_kernel<SB, SRC, EA_CACHE_INT8><<<grid, kCacheThreads, 0, st>>>(a);
    else if constexpr (SB == 64)                        // bf16 has no blocks: cut in 64 rows
        cache_compact_kernel<SB, SRC, EA_CACHE_BF16><<<grid, kCacheThreads, 0, st>>>(a);
}

template <int SB>
static void launch_compact(const CompactArgs &a, dim3 grid, cudaStream_t st)
{
    if (a.src.format == EA_CACHE_BF16)
        launch_compact_src<SB, EA_CACHE_BF16>(a, grid, st);
    else if (a.src.format == EA_CACHE_E4M3)
        launch_compact_src<SB, EA_CACHE_E4M3>(a, grid, st);
    else
        launch_compact_src<SB, EA_CACHE_INT8>(a, grid, st);
}

// Bytes [lo, hi) that K or V of a cache may span.
static void span(const ea_cache *c, const void *p, uintptr_t &lo, uintptr_t &hi)
{
    const int64_t size = c->format == EA_CACHE_BF16 ? 2 : 1;
    const int64_t last = (c->outer - 1) * c->kv_str[0] + (c->rows - 1) * c->kv_str[1] +
                         (c->Hkv - 1) * c->kv_str[2] + c->d;
    lo = reinterpret_cast<uintptr_t>(p);
    hi = lo + static_cast<uintptr_t>(last * size);
}

} // namespace ea

using namespace ea;

extern "C" size_t ea_cache_workspace_size(void) { return sizeof(ea_ws_header); }

extern "C" ea_status ea_cache_write(const ea_cache *c, const void *K_new, const void *V_new,
                                    const int64_t n_str[4], const int32_t *start,
                                    const int32_t *n_new, int B, int T, void *workspace,
                                    size_t ws_bytes, void *stream)
{
    if (!K_new || !V_new || !n_str || T < 1)
        return EA_ERR_INVALID_ARG;
    WriteArgs a{};
    ea_status why;
    if (!cache_dev(c, B, a.c, why))
        return why;
    if (n_str[3] != 1)
        return EA_ERR_INVALID_ARG;
    for (int k = 0; k < 3; ++k)
        if (n_str[k] <= 0 || n_str[k] % 8)
            return EA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(K_new) | reinterpret_cast<uintptr_t>(V_new)) & 15u)
        return EA_ERR_INVALID_ARG;
    const int sb = 1 << a.c.log2sb;
    // new tokens of any length start at any row of a block (bf16 pages need not
    // hold a multiple of the 64 rows used there)
    const int64_t blocks = (static_cast<int64_t>(T) + 2 * sb - 2) / sb;
    if (blocks * a.c.Hkv >= (int64_t(1) << 31))
        return EA_ERR_UNSUPPORTED;
    if (c->format == EA_CACHE_BF16 && c->block_table && c->rows % 64)
        return EA_ERR_UNSUPPORTED;
    if (!ws_ok(workspace, ws_bytes))
        return EA_ERR_WORKSPACE;
    a.x[0] = static_cast<const __nv_bfloat16 *>(K_new);
    a.x[1] = static_cast<const __nv_bfloat16 *>(V_new);
    a.n_sb = n_str[0];
    a.n_st = n_str[1];
    a.n_sh = n_str[2];
    a.start = start;
    a.n_new = n_new;
    a.err = &static_cast<ea_ws_header *>(workspace)->error;
    a.T = T;
    const dim3 grid(static_cast<unsigned>(blocks * a.c.Hkv), static_cast<unsigned>(B), 2);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (a.c.format == EA_CACHE_BF16)
        cache_write_kernel<64, EA_CACHE_BF16><<<grid, kCacheThreads, 0, st>>>(a);
    else if (sb == 16)
        launch_write<16>(a, grid, st);
    else if (sb == 32)
        launch_write<32>(a, grid, st);
    else if (sb == 64)
        launch_write<64>(a, grid, st);
    else
        launch_write<128>(a, grid, st);
    return cudaGetLastError() == cudaSuccess ? EA_OK : EA_ERR_CUDA;
}

extern "C" ea_status ea_cache_compact(const ea_cache *src, const ea_cache *dst,
                                      const int32_t *index, const int32_t *counts, int B, int keep,
                                      const float *weights, float *weights_out, void *workspace,
                                      size_t ws_bytes, void *stream)
{
    if (!index || !counts || keep < 1 || !weights != !weights_out)
        return EA_ERR_INVALID_ARG;
    CompactArgs a{};
    ea_status why;
    if (!cache_dev(src, B, a.src, why) || !cache_dev(dst, B, a.dst, why))
        return why;
    if (a.src.Hkv != a.dst.Hkv || keep > a.dst.cap)
        return EA_ERR_INVALID_ARG;
    if (dst->format == EA_CACHE_BF16 && dst->block_table && dst->rows % 64)
        return EA_ERR_UNSUPPORTED;
    if (!src->block_table || !dst->block_table) {
        for (const void *p : {src->K, src->V})
            for (const void *q : {dst->K, dst->V}) {
                uintptr_t p0, p1, q0, q1;
                span(src, p, p0, p1);
                span(dst, q, q0, q1);
                if (p0 < q1 && q0 < p1)
                    return EA_ERR_INVALID_ARG;
            }
    }
    if (weights) {
        // a row's weight may be read after another row's has been written
        const int64_t rows = static_cast<int64_t>(B) * a.src.Hkv * sizeof(float);
        const uintptr_t w0 = reinterpret_cast<uintptr_t>(weights), o0 = reinterpret_cast<uintptr_t>(weights_out);
        if (w0 < o0 + static_cast<uintptr_t>(rows * a.dst.cap) && o0 < w0 + static_cast<uintptr_t>(rows * a.src.cap))
            return EA_ERR_INVALID_ARG;
    }
    if (!ws_ok(workspace, ws_bytes))
        return EA_ERR_WORKSPACE;
    const int sb = 1 << a.dst.log2sb;
    const int64_t blocks = ceil_div(keep, sb);
    if (blocks * a.dst.Hkv >= (int64_t(1) << 31))
        return EA_ERR_UNSUPPORTED;
    a.index = index;
    a.counts = counts;
    a.w = weights;
    a.w_out = weights_out;
    a.err = &static_cast<ea_ws_header *>(workspace)->error;
    a.keep = keep;
    const dim3 grid(static_cast<unsigned>(blocks * a.dst.Hkv), static_cast<unsigned>(B),
                    a.src.format == EA_CACHE_BF16 ? 2 : 1);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (sb == 16)
        launch_compact<16>(a, grid, st);
    else if (sb == 32)
        launch_compact<32>(a, grid, st);
    else if (sb == 64)
        launch_compact<64>(a, grid, st);
    else
        launch_compact<128>(a, grid, st);
    return cudaGetLastError() == cudaSuccess ? EA_OK : EA_ERR_CUDA;
}

extern "C" ea_status ea_evict_select(const float *weights, const int32_t *seqlens, int B, int Hkv,
                                     int Lmax, int keep, int sink, int recent, int32_t *index,
                                     int32_t *new_seqlens, void *workspace, size_t ws_bytes,
                                     void *stream)
{
    if (!weights || !seqlens || !index || !new_seqlens || B < 1 || Hkv < 1 || Lmax < 1 || keep < 1 ||
        sink < 0 || recent < 0 || static_cast<int64_t>(sink) + recent > keep)
        return EA_ERR_INVALID_ARG;
    if (Lmax > EA_MAX_SEQ || keep > EA_MAX_SEQ || B > 65535 || Hkv > 65535)
        return EA_ERR_UNSUPPORTED;
    if (!ws_ok(workspace, ws_bytes))
        return EA_ERR_WORKSPACE;
    SelectArgs a{};
    a.w = weights;
    a.seqlens = seqlens;
    a.index = index;
    a.new_seqlens = new_seqlens;
    a.err = &static_cast<ea_ws_header *>(workspace)->error;
    a.Hkv = Hkv;
    a.Lmax = Lmax;
    a.keep = keep;
    a.sink = sink;
    a.recent = recent;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return EA_ERR_CUDA;
    const int sms = num_sms(dev);
    if (sms <= 0)
        return EA_ERR_CUDA;
    // CTAs of a (sequence, head): as many as fill the GPU, while each has a few
    // thousand tokens
    int C = 1;
    while (C < kSelMaxCluster && static_cast<int64_t>(B) * Hkv * C * 2 <= 2 * sms && Lmax / (2 * C) >= 2048)
        C *= 2;
    const int share = static_cast<int>(ceil_div(Lmax, C) + 3) & ~3;
    a.cap = share < kSelMaxKeys ? share : kSelMaxKeys;
    const size_t smem = sizeof(SelSmem) + sizeof(uint32_t) * static_cast<size_t>(sel_place(a.cap));
    static bool attr_done[64] = {};   // the attribute is set once per device
    if (dev >= 64 || !attr_done[dev]) {
        if (cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(sizeof(SelSmem) + sizeof(uint32_t) * sel_place(kSelMaxKeys))) != cudaSuccess)
            return EA_ERR_CUDA;
        if (dev < 64)
            attr_done[dev] = true;
    }
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(C);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(C), static_cast<unsigned>(Hkv), static_cast<unsigned>(B));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, evict_select_kernel, a) != cudaSuccess)
        return EA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? EA_OK : EA_ERR_CUDA;
}
