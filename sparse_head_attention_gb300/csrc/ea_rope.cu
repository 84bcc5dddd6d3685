// ea_rope.cu - rotating queries and keys by their positions, alone or on the way
// into a KV cache:
//   y_i = s (x_i cos a - x_j sin a),  y_j = s (x_j cos a + x_i sin a),  a = p f
// for the pairs (i, j) of the first `rot` dims, p the token's position and f the
// pair's frequency.
//
// The angle.  fp32 holds p f to 2^-24 of itself: at p = 10^6 and f = 1 that is 0.06
// rad.  Only a's part of a turn counts, so the kernel works in turns, as fixed point:
// F = frac(f / 2 pi) in units of 2^-64, from f's 24 bits and 128 bits of 1 / 2 pi, and
// p F mod 2^64 is the fraction of a turn of any position, off by p 2^-64 at most.  Its
// upper 32 bits go to sincospif.
//
// A row of a head is 8 threads.  Each holds two runs of 8 dims: both sides of eight
// pairs, or (behind `rot`, and V) dims that only move.  A thread keeps its token's
// eight angles in registers over up to eight heads, where they cost some 10 % of the
// instructions.  Where rows stay bf16 a CTA has 16 tokens, or fewer and more heads; for an
// 8-bit cache it has what is new to one scale block, whose largest rotated value sets the
// scale before the same registers are rounded and stored.  The keys are rounded once, from
// fp32: a key rotated, rounded to bf16 and then quantised would carry two errors.
// (One token of 64 sequences into blocks of 64: 5.4 us; in CTAs of the block's 64 rows,
// and a head group of Q each, 14.4.)
//
// Only data moves, so HBM bounds long inputs (a 32K prefill into bf16 pages, 805 MB: 122 us,
// 0.97 of the measured copy rate; two chunks of 8K, Q and K alone: 55 us, 0.89), and the launch and
// four dependent loads (length, row, page, data) short ones (16 drafts of four sequences 3.4 us).
#include <cuda_runtime.h>

#include "ea_cache.cuh"
#include "ea_internal.h"

namespace ea {

constexpr int kRopeRowThreads = 8;

struct RopeArgs {
    CacheDev c;                          // where has_cache
    const __nv_bfloat16 *x[3];           // Q, K, V
    __nv_bfloat16 *out[2];               // Q, and K without a cache
    int64_t sb[3], st[3], sh[3];         // strides of x
    int64_t ob[2], ot[2], oh[2];         // strides of out
    const float *inv_freq;
    const int32_t *positions, *start, *n_new, *rows;
    uint32_t *err;
    float scale;
    int T, heads[2];                     // Q, K
    int per[2], groups[2], blocks[2];    // heads of a thread, CTAs along the heads, blocks of tokens
    int log2tb;                          // tokens of a CTA where rows stay bf16: few leave room for more heads
    int rot, interleaved, has_cache;
};

// f / 2 pi mod 1 in units of 2^-64; not |f| < 2^24: `bad`.
__device__ __forceinline__ uint64_t turns_per_position(float f, bool &bad)
{
    const uint64_t hi = 0x28be60db9391054aull, lo = 0x7f09d5f47d4d3770ull;    // 1 / 2 pi in units of 2^-128
    const uint32_t u = __float_as_uint(f), e = (u >> 23) & 0xffu;
    const uint64_t m = e ? (u & 0x7fffffu) | 0x800000u : u & 0x7fffffu;
    const int k = 150 - static_cast<int>(e ? e : 1u);                          // |f| = m 2^-k
    bad = k < 0;
    const uint64_t p1 = m * hi + __umul64hi(m, lo);                            // m hi 2^64 + m lo, its upper words
    const uint64_t p2 = __umul64hi(m, hi) + (p1 < m * hi ? 1u : 0u);
    uint64_t t = 0;
    if (k > 0 && k < 64)
        t = p1 >> k | p2 << (64 - k);
    else if (k == 0)
        t = p1;
    else if (k >= 64 && k < 128)
        t = p2 >> (k - 64);
    return (u >> 31) ? 0 - t : t;
}

// A thread's place in a row and its token's angles.
struct Rotation {
    float cs[8], sn[8];
    int a, b;                            // first dims of its two runs
    bool on_a, on_b, pairs_next;         // which of them turn

    __device__ __forceinline__ void place(int j, int rot, int interleaved)
    {
        // (the runs of a row's threads lie side by side, so that each access is of whole sectors: with
        // two neighbouring runs a thread, neighbours and what only moves took 60 and 128 us for 55 and 122)
        const int r16 = rot / 16;
        pairs_next = interleaved != 0;
        if (pairs_next) {
            a = 8 * j;
            b = a + 64;
            on_a = a < rot;
            on_b = b < rot;
        } else {
            on_a = on_b = j < r16;
            a = on_a ? 8 * j : rot + 8 * (j - r16);
            b = a + (on_a ? 8 * r16 : 8 * (8 - r16));
        }
    }
    __device__ __forceinline__ void angles(const float *inv_freq, int j, int pos, float scale)
    {
        if (!on_a)                       // (then not on_b either)
            return;
        const float4 f0 = *reinterpret_cast<const float4 *>(inv_freq + (pairs_next ? 4 : 8) * j);
        const float4 f1 = pairs_next && !on_b ? make_float4(0.f, 0.f, 0.f, 0.f)
                                              : *reinterpret_cast<const float4 *>(inv_freq + (pairs_next ? 4 * j + 32 : 8 * j + 4));
        const float f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            bool bad;
            const uint64_t t = turns_per_position(f[i], bad) * static_cast<uint64_t>(static_cast<int64_t>(pos));
            // half turns, in [-1, 1)
            sincospif(static_cast<float>(static_cast<int32_t>(t >> 32)) * 0x1p-31f, &sn[i], &cs[i]);
            cs[i] = bad ? __uint_as_float(0x7fc00000u) : cs[i] * scale;
            sn[i] = bad ? __uint_as_float(0x7fc00000u) : sn[i] * scale;
        }
    }
    // Neighbours of one run by four of the angles.
    __device__ __forceinline__ void turn_next(float (&u)[8], int k) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = u[2 * i], y = u[2 * i + 1];
            u[2 * i] = fmaf(x, cs[i + k], -(y * sn[i + k]));
            u[2 * i + 1] = fmaf(y, cs[i + k], x * sn[i + k]);
        }
    }
    __device__ __forceinline__ void turn(float (&u)[8], float (&v)[8]) const
    {
        if (pairs_next) {
            if (on_a)
                turn_next(u, 0);
            if (on_b)
                turn_next(v, 4);
        } else if (on_a) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = u[i], y = v[i];
                u[i] = fmaf(x, cs[i], -(y * sn[i]));
                v[i] = fmaf(y, cs[i], x * sn[i]);
            }
        }
    }
};

__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// Rows that stay bf16: heads [h0, h1) of one token, the loads of N in flight.
template <int N>
__device__ __forceinline__ void rope_rows(const __nv_bfloat16 *src, __nv_bfloat16 *dst, int64_t s_sh, int64_t d_sh,
                                          int h0, int h1, const Rotation &r)
{
    for (int h = h0; h < h1; h += N) {
        uint4 raw[N][2];
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (h + k < h1) {
                raw[k][0] = src ? *reinterpret_cast<const uint4 *>(src + (h + k) * s_sh + r.a) : make_uint4(0u, 0u, 0u, 0u);
                raw[k][1] = src ? *reinterpret_cast<const uint4 *>(src + (h + k) * s_sh + r.b) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (h + k < h1) {
                if (r.on_a) {
                    float u[8], v[8];
                    unpack8(raw[k][0], u);
                    unpack8(raw[k][1], v);
                    r.turn(u, v);
                    raw[k][0] = pack8(u);
                    if (r.on_b)          // (what only moves keeps its bits)
                        raw[k][1] = pack8(v);
                }
                *reinterpret_cast<uint4 *>(dst + (h + k) * d_sh + r.a) = raw[k][0];
                *reinterpret_cast<uint4 *>(dst + (h + k) * d_sh + r.b) = raw[k][1];
            }
    }
}

// The input row that new token i of a sequence is; -1 (reported): none of the T.
__device__ __forceinline__ int rope_row(const RopeArgs &a, int b, int i)
{
    if (!a.rows)
        return i;
    const int t = a.rows[static_cast<int64_t>(b) * a.T + i];
    if (t >= 0 && t < a.T)
        return t;
    raise_error(a.err, EA_DEVERR_CHECK);
    return -1;
}

// Threads that an SM holds at least, by the registers of one.  With what they need (88 to 90) CTAs of 512
// threads are alone on an SM: 64 registers (a few spilled) for them, 80 for the smaller ones took a 32K
// prefill from 162 us (blocks of 64), 148 (of 32), 131 (of 16) to 143, 124, 122.  (bf16: 121 with 88, 128 with 80.)
template <int R, int FMT>
constexpr int kRopeResident = FMT == EA_CACHE_BF16 ? 1 : (R <= 32 ? 768 : 1024) / (R * kRopeRowThreads);

// R: rows of a CTA, as many as a scale block of an 8-bit cache has or as tokens come.
template <int R, int FMT>
__global__ void __launch_bounds__(R * kRopeRowThreads, kRopeResident<R, FMT>) rope_kernel(const RopeArgs a)
{
    constexpr bool kQuant = FMT != EA_CACHE_BF16, kE4M3 = FMT == EA_CACHE_E4M3;
    constexpr int kWarps = R * kRopeRowThreads / 32;
    const int b = blockIdx.y;
    // CTAs: Q's blocks of tokens by groups of heads, then K's, then V's
    int x = blockIdx.x, what = 0;
    if (x >= a.blocks[0] * a.groups[0]) {
        x -= a.blocks[0] * a.groups[0];
        what = 1;
        if (x >= a.blocks[1] * a.groups[1]) {
            x -= a.blocks[1] * a.groups[1];
            what = 2;
        }
    }
    const int kind = what ? 1 : 0;
    const int grp = x % a.groups[kind], blk = x / a.groups[kind];
    const int start = a.start ? a.start[b] : 0, n = a.n_new ? a.n_new[b] : a.T;
    if (n < 0 || n > a.T || (a.has_cache && (start < 0 || static_cast<int64_t>(start) + n > a.c.cap))) {
        if (threadIdx.x == 0 && blockIdx.x == 0)
            raise_error(a.err, EA_DEVERR_CHECK);
        return;
    }
    const int r = threadIdx.x / kRopeRowThreads, j = threadIdx.x % kRopeRowThreads;
    const bool cached = what && a.has_cache, rows = !kQuant || !cached;
    const int h0 = (rows ? grp * (R >> a.log2tb) + (r >> a.log2tb) : grp) * a.per[kind];
    const int h1 = min(h0 + a.per[kind], a.heads[kind]);
    Rotation rt;
    rt.place(j, what == 2 ? 0 : a.rot, a.interleaved);
    auto position = [&](int i, int t) {
        return a.positions ? (t >= 0 ? a.positions[static_cast<int64_t>(b) * a.T + t] : 0) : start + i;
    };

    if (rows) {
        const int i = (blk << a.log2tb) + (r & ((1 << a.log2tb) - 1));
        if (i >= n || h0 >= h1)
            return;
        const int t = what ? rope_row(a, b, i) : i;
        __nv_bfloat16 *dst;
        int64_t d_sh;
        if (cached) {
            int outer, row;
            if (!locate(a.c, b, start + i, outer, row, a.err))
                return;
            dst = static_cast<__nv_bfloat16 *>(a.c.code[what - 1]) + outer * a.c.s_outer + row * a.c.s_row;
            d_sh = a.c.s_head;
        } else {
            dst = a.out[what] + b * a.ob[what] + i * a.ot[what];
            d_sh = a.oh[what];
        }
        rt.angles(a.inv_freq, j, position(i, t), a.scale);
        // (two where few registers are left, see kRopeResident; four else: a 32K prefill takes 143 us with two)
        rope_rows<kQuant && R >= 64 ? 2 : 4>(t >= 0 ? a.x[what] + b * a.sb[what] + t * a.st[what] : nullptr, dst, a.sh[what], d_sh, h0, h1, rt);
        return;
    }

    if constexpr (kQuant) {
        __shared__ uint32_t red[2][32];
        const int p0 = ((start >> a.c.log2sb) + blk) << a.c.log2sb;      // the block's first row
        const int lo = max(start, p0), hi = min(start + n, p0 + (1 << a.c.log2sb));
        if (lo >= hi)
            return;
        int outer, row0;
        if (!locate(a.c, b, p0, outer, row0, a.err))
            return;
        const int p = lo + r;                            // (no more than R tokens are new to a block)
        const bool fresh = p < hi;
        const int t = fresh ? rope_row(a, b, p - start) : -1;
        const __nv_bfloat16 *src = a.x[what] + b * a.sb[what] + (t >= 0 ? t : 0) * a.st[what];
        if (fresh)
            rt.angles(a.inv_freq, j, position(p - start, t), a.scale);
        uint8_t *dst = static_cast<uint8_t *>(a.c.code[what - 1]) + outer * a.c.s_outer +
                       row0 * a.c.s_row;
        float *sp = a.c.scale[what - 1] + static_cast<int64_t>(outer) * a.c.Hkv * a.c.nsb + (row0 >> a.c.log2sb);
        uint4 next[2];
        float was_next = 0.f;
        auto load = [&](int h) {
            next[0] = next[1] = make_uint4(0u, 0u, 0u, 0u);
            if (h < h1 && t >= 0) {
                next[0] = *reinterpret_cast<const uint4 *>(src + h * a.sh[what] + rt.a);
                next[1] = *reinterpret_cast<const uint4 *>(src + h * a.sh[what] + rt.b);
            }
            if (h < h1 && lo > p0)
                was_next = sp[static_cast<int64_t>(h) * a.c.nsb];
        };
        load(h0);
        for (int h = h0; h < h1; ++h) {
            float u[8], v[8];
            unpack8(next[0], u);
            unpack8(next[1], v);
            const float was = was_next;
            load(h + 1);
            if (fresh)
                rt.turn(u, v);
            // the largest value of the block (every thread has read the stored scale before
            // the barrier, and it changes behind it)
            uint32_t *rd = red[(h - h0) & 1];
            const uint32_t mine = __reduce_max_sync(0xffffffffu, max(amax8(u), amax8(v)));
            if ((threadIdx.x & 31) == 0)
                rd[threadIdx.x / 32] = mine;
            __syncthreads();
            const int lane = threadIdx.x & 31;
            float s = block_scale(__reduce_max_sync(0xffffffffu, lane < kWarps ? rd[lane] : 0u), kE4M3);
            uint8_t *at = dst + h * a.c.s_head;
            if (lo > p0) {
                // the block already holds rows p0 .. lo - 1
                if (!(was <= s)) {
                    s = isnan(s) ? s : was;              // larger, or NaN: it stays
                } else if (was < s) {
                    const __half2 f = __float2half2_rn(was / s);      // below 1
#pragma unroll 1
                    for (int q = p0 + r; q < lo; q += R)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            uint2 *w = reinterpret_cast<uint2 *>(at + (q - p0) * a.c.s_row + 8 * (2 * j + k));
                            uint32_t c[4];
                            codes_f16<kE4M3>(w->x, c[0], c[1]);
                            codes_f16<kE4M3>(w->y, c[2], c[3]);
                            *w = make_uint2(encode4_f16<kE4M3>(c[0], c[1], f), encode4_f16<kE4M3>(c[2], c[3], f));
                        }
                }
            }
            if (threadIdx.x == 0)
                sp[static_cast<int64_t>(h) * a.c.nsb] = s;
            if (fresh) {
                const bool dead = isnan(s);
                const float inv = dead ? 0.f : 1.f / s;  // a power of two: exact
                uint2 w0 = make_uint2(0u, 0u), w1 = w0;
                if (!dead) {
                    w0 = make_uint2(encode4<kE4M3>(u[0] * inv, u[1] * inv, u[2] * inv, u[3] * inv),
                                    encode4<kE4M3>(u[4] * inv, u[5] * inv, u[6] * inv, u[7] * inv));
                    w1 = make_uint2(encode4<kE4M3>(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                                    encode4<kE4M3>(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
                }
                at += (p - p0) * a.c.s_row;
                *reinterpret_cast<uint2 *>(at + rt.a) = w0;
                *reinterpret_cast<uint2 *>(at + rt.b) = w1;
            }
        }
    }
}

// ------------------------------------------------------------ launches
template <int R>
static void launch_rope_q8(const RopeArgs &a, dim3 grid, cudaStream_t st)
{
    if (a.c.format == EA_CACHE_E4M3)
        rope_kernel<R, EA_CACHE_E4M3><<<grid, R * kRopeRowThreads, 0, st>>>(a);
    else
        rope_kernel<R, EA_CACHE_INT8><<<grid, R * kRopeRowThreads, 0, st>>>(a);
}

static bool rope_tensor(const void *p, const int64_t *str)
{
    if (!p || !str || str[3] != 1 || (reinterpret_cast<uintptr_t>(p) & 15u))
        return false;
    for (int k = 0; k < 3; ++k)
        if (str[k] <= 0 || str[k] % 8)
            return false;
    return true;
}

static void rope_input(RopeArgs &a, int i, const void *p, const int64_t *str)
{
    a.x[i] = static_cast<const __nv_bfloat16 *>(p);
    a.sb[i] = str[0];
    a.st[i] = str[1];
    a.sh[i] = str[2];
}

static void rope_output(RopeArgs &a, int i, void *p, const int64_t *str)
{
    a.out[i] = static_cast<__nv_bfloat16 *>(p);
    a.ob[i] = str[0];
    a.ot[i] = str[1];
    a.oh[i] = str[2];
}

static bool rope_freq(const float *inv_freq, int rot)
{
    return inv_freq && !(reinterpret_cast<uintptr_t>(inv_freq) & 15u) && rot >= 16 && rot <= EA_HEAD_DIM &&
           rot % 16 == 0;
}

// A launch of CTAs of R rows.  A thread's angles serve up to 8 heads, fewer while the threads
// would not fill half of the GPU.  An 8-bit cache's heads follow one another, a barrier each: as few
// of them in a CTA as one wave of CTAs allows (32 accepted paths, e4m3, blocks of 64: 8.0 us with four heads,
// 9.3 with one in three waves).
static ea_status rope_launch(RopeArgs &a, int B, int R, cudaStream_t st)
{
    const bool wide = !a.has_cache || a.c.format == EA_CACHE_BF16;
    // Many queries beside large scale blocks go first and alone, in CTAs of 16 tokens (a 32K prefill into
    // blocks of 64: 131 us in two launches, 143 in one; one token: 7.4 in two, 3.7 in one).
    if (!wide && R >= 64 && ceil_div(a.T, 16) * ceil_div(a.heads[0], 8) * B >= 4 * 152) {
        RopeArgs q = a;
        q.c.format = EA_CACHE_BF16;
        q.heads[1] = 0;
        a.heads[0] = 0;
        const ea_status s = rope_launch(q, B, 16, st);
        if (s != EA_OK)
            return s;
    }
    const int tensors = a.has_cache ? 2 : 1;             // K (and V)
    while ((R >> (a.log2tb + 1)) > 0 && (1 << a.log2tb) < a.T)
        ++a.log2tb;
    const int sub = R >> a.log2tb;
    auto rows = [&](int k, int p) { return static_cast<int64_t>(a.T) * ceil_div(a.heads[k], p) * B; };
    int per = 8;
    while (per > 1 && rows(0, per) + rows(1, per) * tensors < 64 * 152)
        per /= 2;
    a.per[0] = a.per[1] = per;
    a.blocks[0] = a.heads[0] > 0 ? static_cast<int>(ceil_div(a.T, int64_t(1) << a.log2tb)) : 0;
    a.groups[0] = a.heads[0] > 0 ? static_cast<int>(ceil_div(a.heads[0], per * sub)) : 1;
    a.blocks[1] = a.heads[1] > 0 ? static_cast<int>(ceil_div(a.T, int64_t(1) << a.log2tb)) : 0;
    a.groups[1] = a.heads[1] > 0 ? static_cast<int>(ceil_div(a.heads[1], per * sub)) : 1;
    if (!wide) {
        // new tokens of any length start at any row of a scale block
        const int sb = 1 << a.c.log2sb;
        a.blocks[1] = static_cast<int>((static_cast<int64_t>(a.T) + 2 * sb - 2) / sb);
        const int64_t wave = 152 * (R <= 32 ? 768 : 1024) / (R * kRopeRowThreads);
        per = 1;
        while (per < 8 && a.blocks[1] * ceil_div(a.heads[1], per) * tensors * B > wave)
            per *= 2;
        a.per[1] = per;
        a.groups[1] = static_cast<int>(ceil_div(a.heads[1], per));
    }
    const int64_t gx = static_cast<int64_t>(a.blocks[0]) * a.groups[0] +
                       static_cast<int64_t>(a.blocks[1]) * a.groups[1] * tensors;
    if (gx >= (int64_t(1) << 31) || B > 65535)
        return EA_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(B));
    if (wide)
        rope_kernel<16, EA_CACHE_BF16><<<grid, 16 * kRopeRowThreads, 0, st>>>(a);
    else if (R == 16)
        launch_rope_q8<16>(a, grid, st);
    else if (R == 32)
        launch_rope_q8<32>(a, grid, st);
    else if (R == 64)
        launch_rope_q8<64>(a, grid, st);
    else
        launch_rope_q8<128>(a, grid, st);
    return cudaGetLastError() == cudaSuccess ? EA_OK : EA_ERR_CUDA;
}

static bool rope_ws_ok(const void *ws, size_t bytes)
{
    return ws && !(reinterpret_cast<uintptr_t>(ws) & 255u) && bytes >= sizeof(ea_ws_header);
}

} // namespace ea

using namespace ea;

extern "C" ea_status ea_rope(const void *Q, void *Q_out, const int64_t q_str[4], const int64_t qo_str[4], int Hq,
                             const void *K, void *K_out, const int64_t k_str[4], const int64_t ko_str[4], int Hkv,
                             int B, int T, int d, const float *inv_freq, int rot, int interleaved, float rope_scale,
                             const int32_t *positions, const int32_t *n_new, void *workspace, size_t ws_bytes,
                             void *stream)
{
    if (B < 1 || T < 1 || Hq < 0 || Hkv < 0 || (Hq == 0 && Hkv == 0) || !positions || !rope_freq(inv_freq, rot))
        return EA_ERR_INVALID_ARG;
    if (d != EA_HEAD_DIM || B > 65535)
        return EA_ERR_UNSUPPORTED;
    if ((Hq > 0 && (!rope_tensor(Q, q_str) || !rope_tensor(Q_out, qo_str))) ||
        (Hkv > 0 && (!rope_tensor(K, k_str) || !rope_tensor(K_out, ko_str))))
        return EA_ERR_INVALID_ARG;
    if (!rope_ws_ok(workspace, ws_bytes))
        return EA_ERR_WORKSPACE;
    RopeArgs a{};
    if (Hq > 0) {
        rope_input(a, 0, Q, q_str);
        rope_output(a, 0, Q_out, qo_str);
    }
    if (Hkv > 0) {
        rope_input(a, 1, K, k_str);
        rope_output(a, 1, K_out, ko_str);
    }
    a.inv_freq = inv_freq;
    a.positions = positions;
    a.n_new = n_new;
    a.err = &static_cast<ea_ws_header *>(workspace)->error;
    a.scale = rope_scale;
    a.T = T;
    a.heads[0] = Hq;
    a.heads[1] = Hkv;
    a.rot = rot;
    a.interleaved = interleaved != 0;
    return rope_launch(a, B, 16, static_cast<cudaStream_t>(stream));
}

extern "C" ea_status ea_cache_write_rope(const ea_cache *c, const void *K_new, const void *V_new,
                                         const int64_t n_str[4], const void *Q, void *Q_out, const int64_t q_str[4],
                                         const int64_t qo_str[4], int Hq, const float *inv_freq, int rot,
                                         int interleaved, float rope_scale, const int32_t *positions,
                                         const int32_t *start, const int32_t *n_new, const int32_t *rows, int B,
                                         int T, void *workspace, size_t ws_bytes, void *stream)
{
    if (T < 1 || Hq < 0 || (Hq > 0 && rows) || !rope_freq(inv_freq, rot))
        return EA_ERR_INVALID_ARG;
    RopeArgs a{};
    ea_status why;
    if (!cache_dev(c, B, a.c, why))
        return why;
    if (!rope_tensor(K_new, n_str) || !rope_tensor(V_new, n_str) ||
        (Hq > 0 && (!rope_tensor(Q, q_str) || !rope_tensor(Q_out, qo_str))))
        return EA_ERR_INVALID_ARG;
    if (c->format == EA_CACHE_BF16 && c->block_table && c->rows % 64)
        return EA_ERR_UNSUPPORTED;
    if (!rope_ws_ok(workspace, ws_bytes))
        return EA_ERR_WORKSPACE;
    const bool wide = c->format == EA_CACHE_BF16;
    // 16 tokens at most (a decode step's, a path's) take CTAs of 16 rows whatever the block
    const int R = wide || T <= 16 ? 16 : 1 << a.c.log2sb;
    rope_input(a, 1, K_new, n_str);
    rope_input(a, 2, V_new, n_str);
    if (Hq > 0) {
        rope_input(a, 0, Q, q_str);
        rope_output(a, 0, Q_out, qo_str);
    }
    a.inv_freq = inv_freq;
    a.positions = positions;
    a.start = start;
    a.n_new = n_new;
    a.rows = rows;
    a.err = &static_cast<ea_ws_header *>(workspace)->error;
    a.scale = rope_scale;
    a.T = T;
    a.heads[0] = Hq;
    a.heads[1] = a.c.Hkv;
    a.rot = rot;
    a.interleaved = interleaved != 0;
    a.has_cache = 1;
    return rope_launch(a, B, R, static_cast<cudaStream_t>(stream));
}
