// ea_key_weights.cu - the attention weight that the last Tq query rows of each
// sequence give its keys:
//   w[b][h][j] (+)= sum over rows t and the group's heads that keep j of
//                   exp(scale * q_t . k_j - LSE_t),
// with the rows' log-sum-exp given (the prefill and the decode return it), so
// one pass over the products and no softmax statistics are needed.
//
// The products are S^T = K Q^T: keys are the 128 rows of a tcgen05 MMA tile (the
// TMEM lanes) and query rows its columns, so that a thread owns one key and the
// sum over queries is a sum over the columns it reads: no reduction across
// threads, no atomics, one order of summation.  An item is one 128-key tile of a
// (sequence, KV head), or one of `parts` shares of its queries; its key tile is
// loaded once, and the queries' tiles stream past it:
//   warp 0     TMA: K tiles (2 stages of 32 KB) and query tiles (4 of 32 KB)
//   warp 1     the MMAs, into one of four 128-column TMEM buffers
//   warp 2     the rows' LSE, in log2 units, into shared memory
//   warps 4-19 four warpgroups; the one whose buffer is ready reads its columns
//              and adds 2^(s * scale * log2 e - lse)
// A query tile has up to 128 columns.  Where fewer than 65 rows see the key tile
// (a decode step, an observation window) it holds several heads' rows side by
// side, each padded to a multiple of 16, so that one token's step costs one
// 16-column MMA per head and is bound by reading K.  Long rows cost per
// 128 x 128 tile 128^3 multiply-adds (512 cycles of the tensor core) and 16384
// exponentials.
//
// With few key tiles the queries of each are cut into `parts` shares, whose sums
// go to the workspace and are added in order by a last kernel.
#include <cuda.h>
#include <cuda_runtime.h>

#include "ea_device.cuh"
#include "ea_internal.h"

namespace ea {

constexpr int kWTile = 128;                       // keys per tile, query columns per tile
constexpr int kWHalf = kWTile * 128;              // 64 dims of 128 rows: 16 KB
constexpr int kWKStages = 2;
constexpr int kWQStages = 4;
constexpr int kWGroups = 4;                       // warpgroups, TMEM buffers, LSE buffers
constexpr int kWFirstWarp = 4;
constexpr int kWThreads = (kWFirstWarp + 4 * kWGroups) * 32;
constexpr int kWSumThreads = 4 * kWGroups * 32;
constexpr uint32_t kWTmemCols = kWGroups * kWTile;
constexpr int kWMaxParts = 64;

struct __align__(1024) KwSmem {
    uint8_t k[kWKStages][2 * kWHalf];
    uint8_t q[kWQStages][2 * kWHalf];
    float lse[kWGroups][kWTile];
    float red[2][kWGroups][kWTile];
    uint64_t k_full[kWKStages], k_empty[kWKStages];
    uint64_t q_full[kWQStages], q_empty[kWQStages];
    uint64_t s_full[kWGroups], s_free[kWGroups];
    uint64_t lse_full[kWGroups];
    uint64_t item_full[2], item_empty[2];
    int item[2];
    uint32_t tmem_base;
    int abort;
};
constexpr size_t kKwSmemBytes = sizeof(KwSmem) + 1024;
static_assert(kKwSmemBytes <= 232448, "shared memory of one CTA");

struct KwArgs {
    const float *lse;
    int64_t lse_sb, lse_sh;
    const int32_t *seqlens;
    const uint8_t *m, *block_mask;
    float *weights, *partial;
    ea_ws_header *hdr;
    int B, Tq, Lmax, Hkv, g, nB, sink, window, parts, accumulate;
    int n_items;
    float c2;              // scale * log2(e)
};

struct KwItem {
    int b, h, kt, part;
    int L, off;            // query row t sits at position off + t
    int mode;
    int ta, te;            // query rows that see the tile (not EA_BLOCK)
    int s0, s1;            // this share's segments: 128 rows from ta on, or (EA_BLOCK) query blocks
};

// Items: key tile outermost (the first ones are seen by the most queries), then
// share, sequence, head.  False: the sequence has no such tile.
__device__ __forceinline__ bool kw_item(const KwArgs &a, int item, KwItem &x)
{
    const int units = a.B * a.Hkv;
    const int u = item % units, kp = item / units;
    x.part = kp % a.parts;
    x.kt = kp / a.parts;
    x.b = u / a.Hkv;
    x.h = u % a.Hkv;
    x.L = a.seqlens ? a.seqlens[x.b] : a.Lmax;
    if (x.L < 0 || x.L > a.Lmax)
        x.L = 0;
    const int k0 = x.kt * kWTile;
    if (k0 >= x.L)
        return false;
    x.off = x.L - a.Tq;
    x.mode = a.m[u];
    x.ta = max(0, k0 - x.off);
    x.te = a.Tq;
    int n;
    if (x.mode == EA_BLOCK) {
        const int b0 = (x.off + x.ta) / kWTile;              // ta >= -off
        n = a.block_mask ? (x.L - 1) / kWTile + 1 - b0 : 0;
        x.s0 = b0 + static_cast<int>(static_cast<int64_t>(x.part) * n / a.parts);
        x.s1 = b0 + static_cast<int>(static_cast<int64_t>(x.part + 1) * n / a.parts);
        return true;
    }
    if (x.mode == EA_SSA && k0 >= a.sink)                    // the last key's window ends the rows
        x.te = static_cast<int>(min(static_cast<int64_t>(a.Tq),
                                    static_cast<int64_t>(k0) + kWTile - 1 + a.window - x.off));
    n = x.mode > EA_BLOCK ? 0 : max(0, (x.te - x.ta + kWTile - 1) / kWTile);
    x.s0 = static_cast<int>(static_cast<int64_t>(x.part) * n / a.parts);
    x.s1 = static_cast<int>(static_cast<int64_t>(x.part + 1) * n / a.parts);
    return true;
}

// A column tile: rows [t0, t0 + cnt) of heads [head0, head0 + nh) of the group,
// nr columns (cnt rounded up to 16) a head.
struct KwTile {
    int t0, cnt, nr, head0, nh;
};

// Calls f(tile) for every column tile of an item, in order, until f returns
// false; a whole warp calls it.
template <class F>
__device__ __forceinline__ bool kw_tiles(const KwArgs &a, const KwItem &x, int lane, F f)
{
    for (int s = x.s0; s < x.s1; s += 32) {
        uint32_t bits = x.s1 - s >= 32 ? 0xffffffffu : (1u << (x.s1 - s)) - 1u;
        if (x.mode == EA_BLOCK) {
            const int qb = s + lane;
            const int64_t at = ((static_cast<int64_t>(x.b) * a.Hkv + x.h) * a.nB + qb) * a.nB + x.kt;
            bits = __ballot_sync(0xffffffffu, qb < x.s1 && a.block_mask[at] != 0);
        }
        while (bits) {
            const int i = s + __ffs(bits) - 1;
            bits &= bits - 1;
            KwTile t;
            int end;
            if (x.mode == EA_BLOCK) {
                t.t0 = max(i * kWTile - x.off, x.ta);
                end = min((i + 1) * kWTile - x.off, a.Tq);
            } else {
                t.t0 = x.ta + i * kWTile;
                end = min(t.t0 + kWTile, x.te);
            }
            t.cnt = end - t.t0;
            t.nr = (t.cnt + 15) & ~15;
            const int hp = kWTile / t.nr;
            for (t.head0 = 0; t.head0 < a.g; t.head0 += hp) {
                t.nh = min(hp, a.g - t.head0);
                if (!f(t))
                    return false;
            }
        }
    }
    return true;
}

// ------------------------------------------------------------ setup
// Re-arms the queue and reports modes, masks and lengths that cannot be used.
__global__ void __launch_bounds__(256) kw_setup_kernel(const KwArgs a)
{
    bool bad = false;
    for (int u = threadIdx.x; u < a.B * a.Hkv; u += 256) {
        const int mode = a.m[u];
        const int L = a.seqlens ? a.seqlens[u / a.Hkv] : a.Lmax;
        bad |= mode > EA_BLOCK || (mode == EA_BLOCK && !a.block_mask) || L < 0 || L > a.Lmax;
    }
    if (__syncthreads_or(bad) && threadIdx.x == 0)
        raise_error(&a.hdr->error, EA_DEVERR_CHECK);
    if (threadIdx.x == 0)
        a.hdr->work_counter = 0;
}

// ------------------------------------------------------------ roles
// Next item of the queue, handed on in slot it % 2; -1: none left, -2: gave up.
__device__ __forceinline__ int kw_take(const KwArgs &a, KwSmem &sm, int it)
{
    const int slot = it & 1;
    if (!mbar_wait_warp(&sm.item_full[slot], (it >> 1) & 1, &sm.abort, &a.hdr->error))
        return -2;
    const int item = sm.item[slot];
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(&sm.item_empty[slot]);
    return item;
}

__device__ __forceinline__ void kw_producer(const CUtensorMap *tm_k, const CUtensorMap *tm_q,
                                            const CUtensorMap *tm_q16, const KwArgs &a, KwSmem &sm, int lane)
{
    uint32_t *err = &a.hdr->error;
    uint32_t kn = 0, qn = 0;
    bool ok = true;
    for (int it = 0; ok; ++it) {
        const int slot = it & 1;
        if (!mbar_wait_warp(&sm.item_empty[slot], ((it >> 1) & 1) ^ 1, &sm.abort, err))
            break;
        int item = -1;
        KwItem x;
        // tiles that no sequence has are passed over here
        do {
            if (lane == 0) {
                const uint32_t v = atomicAdd(&a.hdr->work_counter, 1u);
                item = v < static_cast<uint32_t>(a.n_items) ? static_cast<int>(v) : -1;
            }
            item = __shfl_sync(0xffffffffu, item, 0);
        } while (item >= 0 && !kw_item(a, item, x));
        if (lane == 0) {
            sm.item[slot] = item;
            mbar_arrive(&sm.item_full[slot]);
        }
        __syncwarp();
        if (item < 0)
            break;
        const int ks = kn % kWKStages;
        if (!mbar_wait_warp(&sm.k_empty[ks], ((kn / kWKStages) & 1) ^ 1, &sm.abort, err))
            break;
        ++kn;
        if (lane == 0) {
            mbar_arrive_expect_tx(&sm.k_full[ks], 2 * kWHalf);
            tma_load_4d(sm.k[ks], tm_k, 0, x.h, x.kt * kWTile, x.b, &sm.k_full[ks]);
            tma_load_4d(sm.k[ks] + kWHalf, tm_k, 64, x.h, x.kt * kWTile, x.b, &sm.k_full[ks]);
        }
        __syncwarp();
        ok = kw_tiles(a, x, lane, [&](const KwTile &t) {
            const int qs = qn % kWQStages;
            if (!mbar_wait_warp(&sm.q_empty[qs], ((qn / kWQStages) & 1) ^ 1, &sm.abort, err))
                return false;
            ++qn;
            if (lane == 0) {
                const int head = x.h * a.g + t.head0;
                mbar_arrive_expect_tx(&sm.q_full[qs], t.nh * t.nr * 256);
                if (t.nr == kWTile) {
                    tma_load_4d(sm.q[qs], tm_q, 0, head, t.t0, x.b, &sm.q_full[qs]);
                    tma_load_4d(sm.q[qs] + kWHalf, tm_q, 64, head, t.t0, x.b, &sm.q_full[qs]);
                } else {
                    int row = 0;
                    for (int hh = 0; hh < t.nh; ++hh)
                        for (int r = 0; r < t.nr; r += 16, row += 16) {
                            tma_load_4d(sm.q[qs] + row * 128, tm_q16, 0, head + hh, t.t0 + r, x.b,
                                        &sm.q_full[qs]);
                            tma_load_4d(sm.q[qs] + kWHalf + row * 128, tm_q16, 64, head + hh, t.t0 + r,
                                        x.b, &sm.q_full[qs]);
                        }
                }
            }
            __syncwarp();
            return true;
        });
    }
    // Before leaving on an abort, let the copies already issued land.
    if (__any_sync(0xffffffffu, *static_cast<volatile int *>(&sm.abort))) {
        volatile int no_abort = 0;
        for (uint32_t k = kn > kWKStages ? kn - kWKStages : 0; k < kn; ++k)
            mbar_wait_warp(&sm.k_full[k % kWKStages], (k / kWKStages) & 1, &no_abort, nullptr);
        for (uint32_t k = qn > kWQStages ? qn - kWQStages : 0; k < qn; ++k)
            mbar_wait_warp(&sm.q_full[k % kWQStages], (k / kWQStages) & 1, &no_abort, nullptr);
    }
}

__device__ __forceinline__ void kw_mma(const KwArgs &a, KwSmem &sm, uint32_t tmem, int lane)
{
    uint32_t *err = &a.hdr->error;
    uint32_t kn = 0, n = 0;
    for (int it = 0;; ++it) {
        const int item = kw_take(a, sm, it);
        if (item < 0)
            break;
        KwItem x;
        kw_item(a, item, x);
        const int ks = kn % kWKStages;
        if (!mbar_wait_warp(&sm.k_full[ks], (kn / kWKStages) & 1, &sm.abort, err))
            break;
        ++kn;
        const uint32_t kaddr = smem_u32(sm.k[ks]);
        const bool ok = kw_tiles(a, x, lane, [&](const KwTile &t) {
            const int buf = n % kWGroups, qs = n % kWQStages;
            if (!mbar_wait_warp(&sm.s_free[buf], ((n / kWGroups) & 1) ^ 1, &sm.abort, err) ||
                !mbar_wait_warp(&sm.q_full[qs], (n / kWQStages) & 1, &sm.abort, err))
                return false;
            ++n;
            tc_fence_after();
            if (lane == 0) {
                const uint32_t idesc = idesc_bf16_f32(kWTile, t.nh * t.nr, false, false);
                const uint32_t qaddr = smem_u32(sm.q[qs]);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t o = (k >> 2) * kWHalf + (k & 3) * 32;
                    tc_mma(tmem + buf * kWTile, sdesc_sw128(kaddr + o, 16, 1024),
                           sdesc_sw128(qaddr + o, 16, 1024), idesc, k > 0 ? 1u : 0u);
                }
                tc_commit(&sm.s_full[buf]);
                tc_commit(&sm.q_empty[qs]);
            }
            __syncwarp();
            return true;
        });
        if (!ok)
            break;
        if (lane == 0)
            tc_commit(&sm.k_empty[ks]);
        __syncwarp();
    }
    // Before leaving on an abort, let the MMAs already issued finish (their
    // operands and accumulators go with the CTA).
    if (__any_sync(0xffffffffu, *static_cast<volatile int *>(&sm.abort)) && n > 0) {
        volatile int no_abort = 0;
        mbar_wait_warp(&sm.s_full[(n - 1) % kWGroups], ((n - 1) / kWGroups) & 1, &no_abort, nullptr);
    }
}

// LSE of each tile's columns in log2 units; rows that keep nothing (-inf) get
// +inf, so that they give 2^-inf = 0.
__device__ __forceinline__ void kw_lse(const KwArgs &a, KwSmem &sm, int lane)
{
    uint32_t *err = &a.hdr->error;
    const float INF = __int_as_float(0x7f800000);
    uint32_t n = 0;
    for (int it = 0;; ++it) {
        const int item = kw_take(a, sm, it);
        if (item < 0)
            break;
        KwItem x;
        kw_item(a, item, x);
        const bool ok = kw_tiles(a, x, lane, [&](const KwTile &t) {
            const int buf = n % kWGroups;
            const float *row = a.lse + x.b * a.lse_sb + (x.h * a.g + t.head0) * a.lse_sh + t.t0;
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = i * 32 + lane, hh = c / t.nr, r = c - hh * t.nr;
                v[i] = hh < t.nh && r < t.cnt ? __ldg(row + hh * a.lse_sh + r) : 0.f;
            }
            if (!mbar_wait_warp(&sm.s_free[buf], ((n / kWGroups) & 1) ^ 1, &sm.abort, err))
                return false;
            ++n;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sm.lse[buf][i * 32 + lane] = v[i] == -INF ? INF : v[i] * 1.4426950408889634f;
            mbar_arrive(&sm.lse_full[buf]);
            return true;
        });
        if (!ok)
            break;
    }
}

// 32 lanes x 16 columns of 32-bit TMEM -> 16 registers per thread.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                   "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr)
                 : "memory");
}

// Barrier of the summing warps that also tells whether any of them failed.
__device__ __forceinline__ bool kw_sync_or(bool failed)
{
    int any;
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "setp.ne.s32 p, %1, 0;\n\t"
                 "barrier.cta.red.or.pred q, 1, %2, p;\n\t"
                 "selp.s32 %0, 1, 0, q;\n\t}"
                 : "=r"(any)
                 : "r"(failed ? 1 : 0), "n"(kWSumThreads)
                 : "memory");
    return any != 0;
}

__device__ __forceinline__ void kw_sum(const KwArgs &a, KwSmem &sm, uint32_t tmem, int warp, int lane)
{
    uint32_t *err = &a.hdr->error;
    const int wg = (warp - kWFirstWarp) >> 2;
    const int key = (warp & 3) * 32 + lane;                  // TMEM lane
    const uint32_t ts = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + wg * kWTile;
    const uint64_t c2 = f2_pack(a.c2, a.c2);
    uint32_t n = 0;                                          // tiles so far, all warpgroups'
    for (int it = 0;; ++it) {
        const int item = kw_take(a, sm, it);
        if (item < 0) {
            kw_sync_or(item == -2);
            return;
        }
        KwItem x;
        kw_item(a, item, x);
        const int j = x.kt * kWTile + key;
        const bool bounded = x.mode == EA_SSA && j >= a.sink;
        float total = 0.f;
        const bool ok = kw_tiles(a, x, lane, [&](const KwTile &t) {
            const uint32_t mine = n++;
            if (static_cast<int>(mine % kWGroups) != wg)
                return true;
            const uint32_t phase = (mine / kWGroups) & 1;
            if (!mbar_wait_warp(&sm.lse_full[wg], phase, &sm.abort, err) ||
                !mbar_wait_warp(&sm.s_full[wg], phase, &sm.abort, err))
                return false;
            tc_fence_after();
            const int cols = t.nh * t.nr;
            // columns [lo, hi) of each head's rows keep key j
            const int i0 = x.off + t.t0;
            const int lo = j - i0;
            const int hi = bounded ? static_cast<int>(min(static_cast<int64_t>(t.cnt),
                                                          static_cast<int64_t>(lo) + a.window))
                                   : t.cnt;
            const bool whole = __all_sync(0xffffffffu, lo <= 0 && hi >= t.nr);
            uint64_t s0 = f2_pack(0.f, 0.f), s1 = s0;
            for (int c = 0; c < cols; c += 16) {
                uint32_t v[16];
                tmem_ld16(ts + c, v);
                tmem_wait_ld();
                const int r0 = c % t.nr;
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const float4 l = *reinterpret_cast<const float4 *>(&sm.lse[wg][c + e]);
                    const uint64_t y0 = f2_fma(f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1])),
                                               c2, f2_pack(-l.x, -l.y));
                    const uint64_t y1 = f2_fma(f2_pack(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])),
                                               c2, f2_pack(-l.z, -l.w));
                    float p[4];
                    f2_unpack(y0, p[0], p[1]);
                    f2_unpack(y1, p[2], p[3]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        p[k] = ex2(p[k]);
                        if (!whole) {
                            const int r = r0 + e + k;
                            p[k] = r >= lo && r < hi ? p[k] : 0.f;
                        }
                    }
                    s0 = f2_add(s0, f2_pack(p[0], p[1]));
                    s1 = f2_add(s1, f2_pack(p[2], p[3]));
                }
            }
            tc_fence_before();
            mbar_arrive(&sm.s_free[wg]);
            float p0, p1;
            f2_unpack(f2_add(s0, s1), p0, p1);
            total += p0 + p1;
            return true;
        });
        float (&red)[kWGroups][kWTile] = sm.red[it & 1];
        red[wg][key] = total;
        if (kw_sync_or(!ok))
            return;
        if (wg == 0 && j < x.L) {
            float w = 0.f;
#pragma unroll
            for (int k = 0; k < kWGroups; ++k)
                w += red[k][key];
            const int64_t at = (static_cast<int64_t>(x.b) * a.Hkv + x.h) * a.Lmax + j;
            if (a.parts > 1)
                a.partial[static_cast<int64_t>(x.part) * a.B * a.Hkv * a.Lmax + at] = w;
            else
                a.weights[at] = a.accumulate ? a.weights[at] + w : w;
        }
    }
}

__global__ void __launch_bounds__(kWThreads, 1)
    key_weights_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_q16, const KwArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    KwSmem &sm = *reinterpret_cast<KwSmem *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kWKStages; ++s) {
            mbar_init(&sm.k_full[s], 1);
            mbar_init(&sm.k_empty[s], 1);
        }
        for (int s = 0; s < kWQStages; ++s) {
            mbar_init(&sm.q_full[s], 1);
            mbar_init(&sm.q_empty[s], 1);
        }
        for (int s = 0; s < kWGroups; ++s) {
            mbar_init(&sm.s_full[s], 1);
            mbar_init(&sm.s_free[s], 128);
            mbar_init(&sm.lse_full[s], 32);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sm.item_full[s], 1);
            mbar_init(&sm.item_empty[s], 2 + 4 * kWGroups);   // MMA, LSE and summing warps
        }
        sm.abort = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == 1) {
        tmem_alloc(&sm.tmem_base, kWTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    if (warp == 0)
        kw_producer(&tm_k, &tm_q, &tm_q16, a, sm, lane);
    else if (warp == 1)
        kw_mma(a, sm, tmem, lane);
    else if (warp == 2)
        kw_lse(a, sm, lane);
    else if (warp >= kWFirstWarp)
        kw_sum(a, sm, tmem, warp, lane);
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kWTmemCols);
    }
}

// Adds the shares of each key in order.
__global__ void __launch_bounds__(256) kw_join_kernel(const KwArgs a)
{
    const int u = blockIdx.y;
    int L = a.seqlens ? a.seqlens[u / a.Hkv] : a.Lmax;
    if (L < 0 || L > a.Lmax)
        L = 0;
    const int j = blockIdx.x * 256 + threadIdx.x;
    if (j >= L)
        return;
    const int64_t at = static_cast<int64_t>(u) * a.Lmax + j;
    const int64_t step = static_cast<int64_t>(a.B) * a.Hkv * a.Lmax;
    float w = 0.f;
#pragma unroll 4
    for (int p = 0; p < a.parts; ++p)
        w += a.partial[p * step + at];
    a.weights[at] = a.accumulate ? a.weights[at] + w : w;
}

// Shares per key tile: enough items for about four per SM of this GPU's 152,
// none shorter than one 128-row segment.  A fixed number of SMs, so that a
// workspace and the result do not depend on the device.
static int kw_parts(int B, int Tq, int Lmax, int Hkv)
{
    const int64_t items = ceil_div(Lmax, kWTile) * B * Hkv;
    const int64_t want = ceil_div(4 * 152, items), most = ceil_div(Tq, kWTile);
    const int64_t p = want < most ? want : most;
    return static_cast<int>(p < 1 ? 1 : p > kWMaxParts ? kWMaxParts : p);
}

} // namespace ea

using namespace ea;

extern "C" size_t ea_key_weights_workspace_size(int B, int Tq, int Lmax, int Hq, int Hkv, int d)
{
    if (B < 1 || Tq < 1 || Lmax < 1 || Lmax > EA_MAX_SEQ || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 ||
        d != EA_HEAD_DIM)
        return 0;
    const int parts = kw_parts(B, Tq, Lmax, Hkv);
    return sizeof(ea_ws_header) +
           (parts > 1 ? align_up(sizeof(float) * static_cast<size_t>(parts) * B * Hkv * Lmax, 256) : 0);
}

extern "C" ea_status ea_key_weights(const void *Q, const void *K, const float *LSE, const int64_t q_str[4],
                                    const int64_t k_str[4], const int64_t lse_str[2],
                                    const int32_t *seqlens, int B, int Tq, int Lmax, int Hq, int Hkv,
                                    int d, float scale, const uint8_t *m, int sink, int window,
                                    const uint8_t *block_mask, int block_size, float *weights,
                                    int accumulate, void *workspace, size_t ws_bytes, void *stream)
{
    if (!Q || !K || !LSE || !q_str || !k_str || !lse_str || !m || !weights || !(scale > 0.f))
        return EA_ERR_INVALID_ARG;
    if (B < 1 || Tq < 1 || Lmax < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || sink < 0 || window < 1 ||
        block_size != EA_TILE)
        return EA_ERR_INVALID_ARG;
    if (d != EA_HEAD_DIM || Lmax > EA_MAX_SEQ || Tq > EA_MAX_SEQ || Hq / Hkv > 64 ||
        static_cast<int64_t>(B) * Hkv > 65535)
        return EA_ERR_UNSUPPORTED;
    if (q_str[3] != 1 || k_str[3] != 1 || lse_str[0] < 0 || lse_str[1] < 0)
        return EA_ERR_INVALID_ARG;
    for (int k = 0; k < 3; ++k)
        if (q_str[k] <= 0 || k_str[k] <= 0 || q_str[k] % 8 || k_str[k] % 8)
            return EA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(Q) | reinterpret_cast<uintptr_t>(K)) & 15u)
        return EA_ERR_INVALID_ARG;
    const size_t need = ea_key_weights_workspace_size(B, Tq, Lmax, Hq, Hkv, d);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || ws_bytes < need)
        return EA_ERR_WORKSPACE;

    KwArgs a{};
    a.lse = LSE;
    a.lse_sb = lse_str[0];
    a.lse_sh = lse_str[1];
    a.seqlens = seqlens;
    a.m = m;
    a.block_mask = block_mask;
    a.weights = weights;
    a.hdr = static_cast<ea_ws_header *>(workspace);
    a.partial = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + sizeof(ea_ws_header));
    a.B = B;
    a.Tq = Tq;
    a.Lmax = Lmax;
    a.Hkv = Hkv;
    a.g = Hq / Hkv;
    a.nB = static_cast<int>(ceil_div(Lmax, EA_TILE));
    a.sink = sink;
    a.window = window;
    a.parts = kw_parts(B, Tq, Lmax, Hkv);
    a.accumulate = accumulate != 0;
    a.c2 = scale * 1.4426950408889634f;
    const int64_t items = static_cast<int64_t>(a.nB) * a.parts * B * Hkv;
    if (items >= (int64_t(1) << 31) - 1024)
        return EA_ERR_UNSUPPORTED;
    a.n_items = static_cast<int>(items);

    alignas(64) CUtensorMap tk, tq, tq16;
    if (!encode_tmap_bf16_4d(&tk, K, d, Hkv, Lmax, B, k_str, 64, kWTile, true) ||
        !encode_tmap_bf16_4d(&tq, Q, d, Hq, Tq, B, q_str, 64, kWTile, true) ||
        !encode_tmap_bf16_4d(&tq16, Q, d, Hq, Tq, B, q_str, 64, 16, true))
        return EA_ERR_INVALID_ARG;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return EA_ERR_CUDA;
    const int sms = num_sms(dev);
    if (sms <= 0)
        return EA_ERR_CUDA;
    static bool attr_done[64] = {};   // the attribute is set once per device
    if (dev >= 64 || !attr_done[dev]) {
        if (cudaFuncSetAttribute(key_weights_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kKwSmemBytes)) != cudaSuccess)
            return EA_ERR_CUDA;
        if (dev < 64)
            attr_done[dev] = true;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    kw_setup_kernel<<<1, 256, 0, st>>>(a);
    key_weights_kernel<<<static_cast<unsigned>(items < sms ? items : sms), kWThreads, kKwSmemBytes, st>>>(
        tk, tq, tq16, a);
    if (a.parts > 1)
        kw_join_kernel<<<dim3(static_cast<unsigned>(ceil_div(Lmax, 256)), static_cast<unsigned>(B * Hkv)), 256,
                         0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? EA_OK : EA_ERR_CUDA;
}
