// ea_key_weights.cu - the attention weight that the last Tq query rows of each
// sequence give its keys:
//   w[b][h][j] (+)= sum over rows t and the group's heads that keep j of
//                   exp(scale * q_t . k_j - LSE_t),
// with the rows' log-sum-exp given (the prefill and the decode return it), so
// one pass over the products and no softmax statistics are needed.
//
// The products are S^T = K Q^T: keys are the 128 rows of a tcgen05 MMA tile (the
// TMEM lanes) and query rows its up to 256 columns, so that a thread owns one
// key and the sum over queries is a sum over the columns it reads: no reduction
// across threads, no atomics, one order of summation.  Roles:
//   warp 0     TMA: key tiles and query tiles
//   warp 1     the MMAs, into two 256-column TMEM buffers
//   warp 2     the rows' LSE as a ninth k-step of the product: -LSE / scale in three
//              bf16 parts (24 bits) in a query's row, against ones in a key's
//   warps 4-19 four warpgroups, two to a buffer: each reads half of its columns
//              and adds 2^(s * scale * log2 e)
// (A summing thread needs every column's LSE.  Read from shared memory beside
// the products, 16 bytes a lane, that took as many of its cycles as the MMAs'
// operands do and paced the kernel: 1200 us for 16K x 16K and 32 heads, 637 with
// nothing summed.)
// A query tile holds 128 rows of two heads (256 rows of one where the group is
// one head), or fewer rows of more heads, each padded to a multiple of 16.
//
// Key tiles go in pairs, one per TMEM buffer, so that a query tile's 64 KB from L2
// feed 2048 cycles of MMAs and the sums over one buffer run under the MMAs into
// the other.  256 columns, because with 128 the operands' reads from shared
// memory pace the MMA (48 % of its cycles busy for 31 % of its rate).
//
// Many rows (more than one query tile per pair): an item is one pair, which stays
// in shared memory while query tiles stream past it in halves of 64 dims (4 stages
// of 32 KB).  Bound by the tensor core (2^22 multiply-adds, 1024 cycles, per 128 x
// 256 tile) and as much by the SFUs (32768 exponentials at 32 a cycle); the chain
// MMA - barrier - sums - barrier over two buffers leaves each at 55 - 60 %.
// Measured: 16384 x 16384 causal, 32 query heads, 842 us (1.1 TFLOP of kept tiles:
// 1.31 PFLOP/s, 0.68 of the measured bf16 rate).
//
// Few rows (a decode step, an observation window): one query tile serves all pairs
// of an item and stays in shared memory; pairs pass through two stages of 64 KB.
// Bound by the same chain, a pair of tiles at a time (about 2 us each), and by the
// launch: 64 rows over 32768 keys, 8 KV heads, 24.5 us (69 MB, 2.8 TB/s).
//
// With few key tiles the queries of each are cut into `parts` shares, whose sums
// go to the workspace and are added in order by a last kernel.
#include <cuda.h>
#include <cuda_runtime.h>

#include "ea_device.cuh"
#include "ea_internal.h"

namespace ea {

constexpr int kWTile = 128;                       // keys per tile
constexpr int kWCols = 256;                       // query columns per tile
constexpr int kWKHalf = kWTile * 128;             // 64 dims of 128 keys: 16 KB
constexpr int kWQHalf = kWCols * 128;             // 64 dims of 256 rows: 32 KB
static_assert(2 * kWKHalf == kWQHalf, "a key tile is as large as half a query tile");
constexpr int kWStages = 4;                       // of 32 KB: many rows, halves of query tiles;
                                                  // few rows, key tiles (two stages of a pair)
constexpr int kWKeys = 2 * kWTile;                // keys of a pair
constexpr int kWXBytes = 32;                      // 16 bf16 of one row of the LSE k-step
constexpr int kWBufs = 2;                         // TMEM and LSE buffers
constexpr int kWGroups = 4;                       // warpgroups, two to a buffer
constexpr int kWFirstWarp = 4;
constexpr int kWThreads = (kWFirstWarp + 4 * kWGroups) * 32;
constexpr int kWSlots = 4;                        // items handed on, and key tiles being joined
constexpr uint32_t kWTmemCols = kWBufs * kWCols;
constexpr int kWMaxParts = 64;

// An item: pairs of key tiles [kt0, kt1) of one (sequence, KV head) and one share
// of their queries.
struct KwItem {
    int valid;             // 0: none left
    int b, h, part, kt0, kt1;
    int L, off;            // query row t sits at position off + t
    int mode;
};

struct __align__(1024) KwSmem {
    uint8_t held[2 * kWQHalf];                    // many rows: two key tiles; few rows: a query tile
    uint8_t ring[kWStages][kWQHalf];
    uint8_t qx[kWBufs][kWXBytes * kWCols];        // the LSE k-step: query rows
    uint8_t kx[kWXBytes * kWTile];                // and key rows (ones)
    float red[kWBufs][kWSlots][kWTile];
    uint64_t k_full[kWStages], k_empty[kWStages];
    uint64_t q_full[kWStages], q_empty[kWStages];
    uint64_t s_full[kWBufs], s_free[kWBufs];
    uint64_t lse_full[kWBufs], lse_empty[kWBufs];
    uint64_t red_full[kWBufs][kWSlots], red_empty[kWBufs][kWSlots];
    uint64_t item_full[kWSlots], item_empty[kWSlots];
    uint64_t drain;
    KwItem item[kWSlots];
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
    int B, Tq, Lmax, Hkv, g, nB, sink, window, parts, run, accumulate;
    int seg, seg_log2;     // query rows of one head in a tile: 128, or 256 for groups of one head
    int box;               // rows of a query box: 128, or all of Tq (rounded up to 16)
    int n_items;
    int one_each;          // an item or none for each CTA: no queue
    float c2;              // scale * log2(e)
    float inv_scale;
};

// Items: runs of pairs outermost (the first ones are seen by the most
// queries), then share, sequence, head.  False: the sequence has no such tile.
__device__ __forceinline__ bool kw_item(const KwArgs &a, int item, KwItem &x)
{
    const int units = a.B * a.Hkv;
    const int u = item % units, kp = item / units;
    x.part = kp % a.parts;
    x.kt0 = kp / a.parts * a.run;
    x.b = u / a.Hkv;
    x.h = u % a.Hkv;
    x.L = a.seqlens ? a.seqlens[x.b] : a.Lmax;
    if (x.L < 0 || x.L > a.Lmax)
        x.L = 0;
    x.kt1 = min(x.kt0 + a.run, (x.L + kWKeys - 1) / kWKeys);
    x.off = x.L - a.Tq;
    x.mode = a.m[u];
    x.valid = 1;
    return x.kt0 < x.kt1;
}

// The queries of one pair that an item takes.
struct KwRange {
    int ta, te;            // query rows that see the pair (not EA_BLOCK: te)
    int s0, s1;            // this share's segments: a.seg rows from ta on, or (EA_BLOCK) query blocks
};

__device__ __forceinline__ KwRange kw_range(const KwArgs &a, const KwItem &x, int kt)
{
    KwRange r;
    const int k0 = kt * kWKeys;
    r.ta = max(0, k0 - x.off);
    r.te = a.Tq;
    int n, first = 0;
    if (x.mode == EA_BLOCK) {
        first = (x.off + r.ta) / kWTile;                     // ta >= -off
        n = a.block_mask ? (x.L - 1) / kWTile + 1 - first : 0;
    } else {
        if (x.mode == EA_SSA && k0 >= a.sink)                // the last key's window ends the rows
            r.te = min(a.Tq, k0 + kWKeys - 1 + a.window - x.off);
        n = x.mode > EA_BLOCK || r.te <= r.ta ? 0 : (r.te - r.ta + a.seg - 1) >> a.seg_log2;
    }
    r.s0 = first;
    r.s1 = first + n;
    if (a.parts > 1) {                                       // n <= 2^14, parts <= 64
        r.s0 = first + x.part * n / a.parts;
        r.s1 = first + (x.part + 1) * n / a.parts;
    }
    return r;
}

// A column tile: rows [t0, t0 + cnt) of heads [head0, head0 + nh) of the group,
// nr columns (cnt rounded up to 16) a head.
struct KwTile {
    int t0, cnt, nr, head0, nh;
    uint32_t keep;         // bit p: the rows' block keeps key tile p of a pair (EA_BLOCK)
};

// Heads of nr columns (16 .. 256, in sixteens) that fit a tile: 256 / nr, without
// a division (the roles' integer code runs at one warp's pace, between MMAs).
__device__ __forceinline__ int kw_heads(int nr)
{
    return static_cast<int>((0x1112347Full >> (nr / 4 - 4)) & 15u) + 1;
}

// Calls f(tile) for every column tile of a pair, in order, until f returns
// false; a whole warp calls it.
template <class F>
__device__ __forceinline__ bool kw_tiles(const KwArgs &a, const KwItem &x, const KwRange &rg, int kt,
                                         int lane, F f)
{
    for (int s = rg.s0; s < rg.s1; s += 32) {
        uint32_t bits = rg.s1 - s >= 32 ? 0xffffffffu : (1u << (rg.s1 - s)) - 1u;
        uint32_t bits0 = bits, bits1 = bits;
        if (x.mode == EA_BLOCK) {
            const int qb = s + lane, kb = 2 * kt;
            const uint8_t *row = a.block_mask +
                                 ((static_cast<int64_t>(x.b) * a.Hkv + x.h) * a.nB + qb) * a.nB + kb;
            bits0 = __ballot_sync(0xffffffffu, qb < rg.s1 && row[0] != 0);
            bits1 = __ballot_sync(0xffffffffu, qb < rg.s1 && kb + 1 < a.nB && row[1] != 0);
            bits = bits0 | bits1;
        }
        while (bits) {
            const int bit = __ffs(bits) - 1, i = s + bit;
            bits &= bits - 1;
            KwTile t;
            t.keep = ((bits0 >> bit) & 1u) | ((bits1 >> bit) & 1u) << 1;
            int end;
            if (x.mode == EA_BLOCK) {
                t.t0 = max(i * kWTile - x.off, rg.ta);
                end = min((i + 1) * kWTile - x.off, a.Tq);
            } else {
                t.t0 = rg.ta + i * a.seg;
                end = min(t.t0 + a.seg, rg.te);
            }
            t.cnt = end - t.t0;
            t.nr = (t.cnt + 15) & ~15;
            const int hp = kw_heads(t.nr);
            for (t.head0 = 0; t.head0 < a.g; t.head0 += hp) {
                t.nh = min(hp, a.g - t.head0);
                if (!f(t))
                    return false;
            }
        }
    }
    return true;
}

// A query tile held in shared memory, followed alike by the producer and the MMA
// warp (its LSE by its warp): a tile equal to the one before it is not loaded again.
struct KwHeld {
    int b, h, t0, cnt, head0;
    uint32_t n;            // query tiles loaded
    __device__ __forceinline__ bool same(const KwItem &x, const KwTile &t)
    {
        const bool eq = n > 0 && b == x.b && h == x.h && t0 == t.t0 && cnt == t.cnt && head0 == t.head0;
        b = x.b;
        h = x.h;
        t0 = t.t0;
        cnt = t.cnt;
        head0 = t.head0;
        return eq;
    }
};

// ------------------------------------------------------------ setup
// Reports modes, masks and lengths that cannot be used (threads first, first + step, ...).
__device__ __forceinline__ void kw_check(const KwArgs &a, int first, int step)
{
    bool bad = false;
    for (int u = first; u < a.B * a.Hkv; u += step) {
        const int mode = a.m[u];
        const int L = a.seqlens ? a.seqlens[u / a.Hkv] : a.Lmax;
        bad |= mode > EA_BLOCK || (mode == EA_BLOCK && !a.block_mask) || L < 0 || L > a.Lmax;
    }
    if (bad)
        raise_error(&a.hdr->error, EA_DEVERR_CHECK);
}

// Re-arms the queue.  With an item for each CTA at most there is none, and a warp of
// the first CTA checks (64 rows over 32K keys 26.9 -> 24.5 us).
__global__ void __launch_bounds__(256) kw_setup_kernel(const KwArgs a)
{
    griddep_launch_dependents();   // the products' kernel may start its prologue
    kw_check(a, threadIdx.x, 256);
    if (threadIdx.x == 0)
        a.hdr->work_counter = 0;
}

// ------------------------------------------------------------ roles
// Next item of the queue (slot it % kWSlots); 0: none left, -1: gave up.
__device__ __forceinline__ int kw_take(const KwArgs &a, KwSmem &sm, int it, KwItem &x)
{
    const int slot = it % kWSlots;
    if (!mbar_wait_warp(&sm.item_full[slot], (it / kWSlots) & 1, &sm.abort, &a.hdr->error))
        return -1;
    x = sm.item[slot];
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(&sm.item_empty[slot]);
    return x.valid;
}

// The query tiles' tensor maps: boxes of 64 dims x `rows` rows, and of 16 rows for
// tiles that are not whole boxes.  (A copy takes its issuing thread about 240
// cycles: 32 boxes of 16 rows for one tile cost more than the tile's MMAs.)
struct KwMaps {
    CUtensorMap rows, r16;
};

// Dims 64 half .. + 63 of a query tile's rows, into dst.
__device__ __forceinline__ void kw_load_q(const KwMaps &tm, const KwArgs &a, uint8_t *dst, int head, int b,
                                          const KwTile &t, int half, uint64_t *bar)
{
    const bool whole = t.nr == a.box || (t.nr == kWCols && a.box == kWTile);
    const int box = whole ? a.box : 16;
    const CUtensorMap *map = whole ? &tm.rows : &tm.r16;
    int row = 0;
    for (int hh = 0; hh < t.nh; ++hh)
        for (int r = 0; r < t.nr; r += box, row += box)
            tma_load_4d(dst + row * 128, map, 64 * half, head + hh, t.t0 + r, b, bar);
}

// A ring position: stage and phase.
template <int N>
struct KwRing {
    int s = 0;
    uint32_t phase = 0;
    uint32_t n = 0;        // steps taken
    __device__ __forceinline__ void next()
    {
        ++n;
        if (++s == N) {
            s = 0;
            phase ^= 1;
        }
    }
};

template <bool MANY>
__device__ __forceinline__ void kw_producer(const CUtensorMap *tm_k, const KwMaps &tm_q, const KwArgs &a, KwSmem &sm, int lane)
{
    uint32_t *err = &a.hdr->error;
    constexpr int KS = MANY ? 1 : kWStages / 2, QS = MANY ? kWStages : 1;
    KwRing<KS> k;
    KwRing<QS> q;
    KwHeld held{};
    bool ok = true;
    uint32_t own = blockIdx.x;                               // one_each: this CTA's item, then none
    auto draw = [&]() {
        if (a.one_each) {
            const uint32_t v = own;
            own = 0xffffffffu;
            return v;
        }
        return lane == 0 ? atomicAdd(&a.hdr->work_counter, 1u) : 0u;
    };
    uint32_t next = draw();                                  // drawn an item ahead
    for (int it = 0; ok; ++it) {
        const int slot = it % kWSlots;
        KwItem x{};
        // runs that no sequence reaches are passed over here
        while (true) {
            const uint32_t v = __shfl_sync(0xffffffffu, next, 0);
            x.valid = 0;
            if (v >= static_cast<uint32_t>(a.n_items))
                break;
            next = draw();
            if (kw_item(a, static_cast<int>(v), x))
                break;
        }
        if (!mbar_wait_warp(&sm.item_empty[slot], ((it / kWSlots) & 1) ^ 1, &sm.abort, err))
            break;
        if (lane == 0) {
            sm.item[slot] = x;
            mbar_arrive(&sm.item_full[slot]);
        }
        __syncwarp();
        if (!x.valid)
            break;
        for (int kt = x.kt0; ok && kt < x.kt1; ++kt) {
            const KwRange rg = kw_range(a, x, kt);
            if (rg.s0 >= rg.s1)
                continue;
            if (!mbar_wait_warp(&sm.k_empty[k.s], k.phase ^ 1, &sm.abort, err)) {
                ok = false;
                break;
            }
            if (lane == 0) {
                mbar_arrive_expect_tx(&sm.k_full[k.s], 4 * kWKHalf);
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    uint8_t *dst = MANY ? sm.held + p * 2 * kWKHalf : sm.ring[2 * k.s + p];
                    const int row = kt * kWKeys + p * kWTile;
                    tma_load_4d(dst, tm_k, 0, x.h, row, x.b, &sm.k_full[k.s]);
                    tma_load_4d(dst + kWKHalf, tm_k, 64, x.h, row, x.b, &sm.k_full[k.s]);
                }
            }
            __syncwarp();
            k.next();
            ok = kw_tiles(a, x, rg, kt, lane, [&](const KwTile &t) {
                const int head = x.h * a.g + t.head0;
                if constexpr (MANY) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        if (!mbar_wait_warp(&sm.q_empty[q.s], q.phase ^ 1, &sm.abort, err))
                            return false;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&sm.q_full[q.s], t.nh * t.nr * 128);
                            kw_load_q(tm_q, a, sm.ring[q.s], head, x.b, t, half, &sm.q_full[q.s]);
                        }
                        __syncwarp();
                        q.next();
                    }
                } else if (!held.same(x, t)) {
                    if (!mbar_wait_warp(&sm.q_empty[q.s], q.phase ^ 1, &sm.abort, err))
                        return false;
                    ++held.n;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&sm.q_full[q.s], t.nh * t.nr * 256);
                        kw_load_q(tm_q, a, sm.held, head, x.b, t, 0, &sm.q_full[q.s]);
                        kw_load_q(tm_q, a, sm.held + kWQHalf, head, x.b, t, 1, &sm.q_full[q.s]);
                    }
                    __syncwarp();
                    q.next();
                }
                return true;
            });
        }
    }
    // Before leaving on an abort, let the copies already issued land.
    if (__any_sync(0xffffffffu, *static_cast<volatile int *>(&sm.abort))) {
        volatile int no_abort = 0;
        for (uint32_t n = k.n > KS ? k.n - KS : 0; n < k.n; ++n)
            mbar_wait_warp(&sm.k_full[n % KS], (n / KS) & 1, &no_abort, nullptr);
        for (uint32_t n = q.n > QS ? q.n - QS : 0; n < q.n; ++n)
            mbar_wait_warp(&sm.q_full[n % QS], (n / QS) & 1, &no_abort, nullptr);
    }
}

// The LSE k-step's operands are stored without swizzle: 8 rows x 16 bytes of a
// core matrix follow one another, the two along k are 128 bytes apart, the next
// eight rows 256.
__device__ __forceinline__ uint64_t kw_sdesc_x(uint32_t saddr)
{
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(128 >> 4) << 16 |
           static_cast<uint64_t>(256 >> 4) << 32 | static_cast<uint64_t>(1) << 46;
}

__device__ __forceinline__ uint8_t *kw_row_x(uint8_t *base, int row)
{
    return base + (row >> 3) * 256 + (row & 7) * 16;
}

// The MMAs of both key tiles of a pair, one after the other, so that the first
// one's sums run under the second one's MMAs.  (Alternating between them every 64
// dims ended both together and left MMAs and exponentials to take turns: 1091 us
// for 16K x 16K and 32 heads against 850; a warp each, in turns by a token: 945.)
template <bool MANY>
__device__ __forceinline__ void kw_mma(const KwArgs &a, KwSmem &sm, uint32_t tmem, int lane)
{
    uint32_t *err = &a.hdr->error;
    constexpr int KS = MANY ? 1 : kWStages / 2, QS = MANY ? kWStages : 1;
    KwRing<KS> k;
    KwRing<QS> q;
    uint32_t n = 0;                                          // column tiles
    const uint32_t ring = smem_u32(sm.ring[0]), held_addr = smem_u32(sm.held);
    const uint64_t kx = kw_sdesc_x(smem_u32(sm.kx));
    KwHeld held{};
    bool ok = true;
    KwItem x;
    // the nine MMAs of a tile: 2 x 64 dims and the LSE
    auto mma = [&](uint32_t d, uint32_t ka, uint32_t qa, uint32_t qx, uint32_t idesc) {
        const uint64_t k0 = sdesc_sw128(ka, 16, 1024), k1 = sdesc_sw128(ka + kWKHalf, 16, 1024);
        const uint64_t q0 = sdesc_sw128(qa, 16, 1024), q1 = sdesc_sw128(qa + kWQHalf, 16, 1024);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            tc_mma(d, k0 + 2 * i, q0 + 2 * i, idesc, i == 0 ? 0u : 1u);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            tc_mma(d, k1 + 2 * i, q1 + 2 * i, idesc, 1u);
        tc_mma(d, kx, kw_sdesc_x(qx), idesc, 1u);
    };
    for (int it = 0; ok && kw_take(a, sm, it, x) > 0; ++it) {
        for (int kt = x.kt0; ok && kt < x.kt1; ++kt) {
            const KwRange rg = kw_range(a, x, kt);
            if (rg.s0 >= rg.s1)
                continue;
            ok = mbar_wait_warp(&sm.k_full[k.s], k.phase, &sm.abort, err);
            if (!ok)
                break;
            const uint32_t kaddr = MANY ? held_addr : ring + k.s * 2 * kWQHalf;
            ok = kw_tiles(a, x, rg, kt, lane, [&](const KwTile &t) {
                const uint32_t idesc = idesc_bf16_f32(kWTile, t.nh * t.nr, false, false);
                const uint32_t mine = n++;
                const int lb = mine % kWBufs;
                const uint32_t qa = MANY ? ring + q.s * kWQHalf : held_addr, qx = smem_u32(sm.qx[lb]);
                if constexpr (MANY) {
                    if (!mbar_wait_warp(&sm.q_full[q.s], q.phase, &sm.abort, err) ||
                        !mbar_wait_warp(&sm.q_full[q.s + 1], q.phase, &sm.abort, err))
                        return false;
                } else if (!held.same(x, t)) {
                    // the tile before it is done with once the MMAs so far are
                    if (held.n > 0) {
                        if (lane == 0)
                            tc_commit(&sm.q_empty[0]);
                        __syncwarp();
                        q.next();
                    }
                    if (!mbar_wait_warp(&sm.q_full[0], q.phase, &sm.abort, err))
                        return false;
                    ++held.n;
                }
                if (!mbar_wait_warp(&sm.lse_full[lb], (mine / kWBufs) & 1, &sm.abort, err))
                    return false;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    if (!mbar_wait_warp(&sm.s_free[b], (mine & 1) ^ 1, &sm.abort, err))
                        return false;
                    tc_fence_after();
                    if (lane == 0) {
                        mma(tmem + b * kWCols, kaddr + b * 2 * kWKHalf, qa, qx, idesc);
                        tc_commit(&sm.s_full[b]);
                        if (b == 1) {
                            if constexpr (MANY) {
                                tc_commit(&sm.q_empty[q.s]);
                                tc_commit(&sm.q_empty[q.s + 1]);
                            }
                            tc_commit(&sm.lse_empty[lb]);
                        }
                    }
                    __syncwarp();
                }
                if constexpr (MANY) {
                    q.next();
                    q.next();                            // two halves: q.s is 0 or 2
                }
                return true;
            });
            if (ok && lane == 0)
                tc_commit(&sm.k_empty[k.s]);
            __syncwarp();
            k.next();
        }
    }
    // Before leaving on an abort, let the MMAs already issued finish (their
    // operands and accumulators go with the CTA): a commit on a barrier of their
    // own covers them.
    if (__any_sync(0xffffffffu, *static_cast<volatile int *>(&sm.abort)) && n > 0) {
        volatile int no_abort = 0;
        if (lane == 0)
            tc_commit(&sm.drain);
        __syncwarp();
        mbar_wait_warp(&sm.drain, 0, &no_abort, nullptr);
    }
}

// -LSE / scale of each tile's columns, in three bf16 parts whose sum is the fp32
// value; rows that keep nothing (LSE = -inf) get -inf, so that they give
// 2^-inf = 0.
template <bool MANY>
__device__ __forceinline__ void kw_lse(const KwArgs &a, KwSmem &sm, int lane)
{
    uint32_t *err = &a.hdr->error;
    const float INF = __int_as_float(0x7f800000);
    KwRing<kWBufs> buf;
    bool ok = true;
    KwItem x;
    KwHeld held[kWBufs] = {};                                // n: 1 once the buffer holds a tile's
    for (int it = 0; ok && kw_take(a, sm, it, x) > 0; ++it)
        for (int kt = x.kt0; ok && kt < x.kt1; ++kt)
            ok = kw_tiles(a, x, kw_range(a, x, kt), kt, lane, [&](const KwTile &t) {
                const bool same = !MANY && (buf.s ? held[1].same(x, t) : held[0].same(x, t));
                float v[kWCols / 32];
                if (!same) {
                    held[0].n |= buf.s == 0;
                    held[1].n |= buf.s == 1;
                    const float *row = a.lse + x.b * a.lse_sb + (x.h * a.g + t.head0) * a.lse_sh + t.t0;
                    if (t.nr == kWTile) {
#pragma unroll
                        for (int i = 0; i < kWCols / 32; ++i) {
                            const int hh = i / 4, r = i % 4 * 32 + lane;
                            v[i] = hh < t.nh && r < t.cnt ? __ldg(row + hh * a.lse_sh + r) : 0.f;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < kWCols / 32; ++i) {
                            const int c = i * 32 + lane, hh = c / t.nr, r = c - hh * t.nr;
                            v[i] = hh < t.nh && r < t.cnt ? __ldg(row + hh * a.lse_sh + r) : 0.f;
                        }
                    }
                }
                if (!mbar_wait_warp(&sm.lse_empty[buf.s], buf.phase ^ 1, &sm.abort, err))
                    return false;
                if (!same) {
#pragma unroll
                    for (int i = 0; i < kWCols / 32; ++i) {
                        const float f = v[i] == -INF ? -INF : v[i] * -a.inv_scale;
                        const float hi = __bfloat162float(__float2bfloat16_rn(f));
                        const float r1 = fabsf(f) < INF && fabsf(hi) < INF ? f - hi : 0.f;
                        const float mid = __bfloat162float(__float2bfloat16_rn(r1));
                        *reinterpret_cast<uint4 *>(kw_row_x(sm.qx[buf.s], i * 32 + lane)) =
                            make_uint4(pack_bf16x2(hi, mid), pack_bf16x2(r1 - mid, 0.f), 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                mbar_arrive(&sm.lse_full[buf.s]);
                buf.next();
                return true;
            });
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

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Adds 2^(v * c2) over N columns to two pairs of sums; with MASKED only the
// columns e with lo <= e < hi.
template <int N, bool MASKED>
__device__ __forceinline__ void kw_add(const uint32_t (&v)[N], uint64_t c2, int lo, int hi, uint64_t &s0,
                                       uint64_t &s1)
{
#pragma unroll
    for (int e = 0; e < N; e += 4) {
        float p[4];
        f2_unpack(f2_mul(f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), c2), p[0], p[1]);
        f2_unpack(f2_mul(f2_pack(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])), c2), p[2], p[3]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            p[k] = ex2(p[k]);
            if (MASKED)
                p[k] = e + k >= lo && e + k < hi ? p[k] : 0.f;
        }
        s0 = f2_add(s0, f2_pack(p[0], p[1]));
        s1 = f2_add(s1, f2_pack(p[2], p[3]));
    }
}

// The columns [c0, c1) of one key tile's products: thread sums, rows [lo, hi) of
// each head.  ts: the buffer's TMEM address at this warp's lanes.
__device__ __forceinline__ float kw_columns(uint32_t ts, int c0, int c1, int nr, int lo, int hi, uint64_t c2)
{
    uint64_t s0 = f2_pack(0.f, 0.f), s1 = s0;
    if (__all_sync(0xffffffffu, lo <= 0 && hi >= nr)) {
        int c = c0;
        for (; c + 64 <= c1; c += 64) {
            // the second load runs under the first one's sums
            uint32_t v0[32], v1[32];
            tmem_ld32(ts + c, v0);
            tmem_wait_ld();
            tmem_ld32(ts + c + 32, v1);
            kw_add<32, false>(v0, c2, 0, 0, s0, s1);
            tmem_wait_ld();
            kw_add<32, false>(v1, c2, 0, 0, s0, s1);
        }
        for (; c < c1; c += 16) {
            uint32_t v[16];
            tmem_ld16(ts + c, v);
            tmem_wait_ld();
            kw_add<16, false>(v, c2, 0, 0, s0, s1);
        }
    } else if (__any_sync(0xffffffffu, lo < hi)) {
        for (int c = c0; c < c1; c += 16) {
            uint32_t v[16];
            tmem_ld16(ts + c, v);
            tmem_wait_ld();
            const int r0 = c % nr;
            kw_add<16, true>(v, c2, lo - r0, hi - r0, s0, s1);
        }
    }
    float p0, p1;
    f2_unpack(f2_add(s0, s1), p0, p1);
    return p0 + p1;
}

__device__ __forceinline__ void kw_sum(const KwArgs &a, KwSmem &sm, uint32_t tmem, int warp, int lane)
{
    uint32_t *err = &a.hdr->error;
    const int wg = (warp - kWFirstWarp) >> 2;
    const int buf = wg >> 1, half = wg & 1;                  // key tile of the pair, half of the columns
    const int key = (warp & 3) * 32 + lane;                  // TMEM lane
    const uint32_t ts = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + buf * kWCols;
    const uint64_t c2 = f2_pack(a.c2, a.c2);
    uint32_t n = 0, kc = 0;                                  // column tiles and pairs so far
    bool ok = true;
    KwItem x;
    for (int it = 0; ok && kw_take(a, sm, it, x) > 0; ++it) {
        for (int kt = x.kt0; ok && kt < x.kt1; ++kt) {
            const KwRange rg = kw_range(a, x, kt);
            const int j = kt * kWKeys + buf * kWTile + key;
            const bool bounded = x.mode == EA_SSA && j >= a.sink;
            float total = 0.f;
            ok = kw_tiles(a, x, rg, kt, lane, [&](const KwTile &t) {
                if (!mbar_wait_warp(&sm.s_full[buf], n & 1, &sm.abort, err))
                    return false;
                ++n;
                tc_fence_after();
                const int q16 = t.nh * t.nr / 16, mid = 16 * ((q16 + 1) / 2);
                // rows [lo, hi) of each head keep key j
                const int lo = j - (x.off + t.t0);
                int hi = bounded ? min(t.cnt, lo + a.window) : t.cnt;
                if (!((t.keep >> buf) & 1u))
                    hi = 0;
                const float w = kw_columns(ts, half ? mid : 0, half ? 16 * q16 : mid, t.nr, lo, hi, c2);
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sm.s_free[buf]);
                total += w;
                return true;
            });
            if (!ok)
                break;
            // the two warpgroups' sums are joined by the first
            const int slot = kc % kWSlots;
            const uint32_t phase = (kc / kWSlots) & 1;
            ++kc;
            if (half) {
                ok = mbar_wait_warp(&sm.red_empty[buf][slot], phase ^ 1, &sm.abort, err);
                if (!ok)
                    break;
                sm.red[buf][slot][key] = total;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sm.red_full[buf][slot]);
                continue;
            }
            ok = mbar_wait_warp(&sm.red_full[buf][slot], phase, &sm.abort, err);
            if (!ok)
                break;
            const float w = total + sm.red[buf][slot][key];
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sm.red_empty[buf][slot]);
            if (j < x.L) {
                const int64_t at = (static_cast<int64_t>(x.b) * a.Hkv + x.h) * a.Lmax + j;
                if (a.parts > 1)
                    a.partial[static_cast<int64_t>(x.part) * a.B * a.Hkv * a.Lmax + at] = w;
                else
                    a.weights[at] = a.accumulate ? a.weights[at] + w : w;
            }
        }
    }
}

template <bool MANY>
__global__ void __launch_bounds__(kWThreads, 1)
    key_weights_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ KwMaps tm_q,
                       const KwArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    KwSmem &sm = *reinterpret_cast<KwSmem *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kWStages; ++s) {
            mbar_init(&sm.k_full[s], 1);
            mbar_init(&sm.k_empty[s], 1);
            mbar_init(&sm.q_full[s], 1);
            mbar_init(&sm.q_empty[s], 1);
        }
        for (int s = 0; s < kWBufs; ++s) {
            mbar_init(&sm.s_full[s], 1);
            mbar_init(&sm.s_free[s], 8);                      // the warps of a buffer's warpgroups
            mbar_init(&sm.lse_full[s], 32);
            mbar_init(&sm.lse_empty[s], 1);
        }
        for (int s = 0; s < kWSlots; ++s) {
            for (int b = 0; b < kWBufs; ++b) {
                mbar_init(&sm.red_full[b][s], 4);
                mbar_init(&sm.red_empty[b][s], 4);
            }
            mbar_init(&sm.item_full[s], 1);
            mbar_init(&sm.item_empty[s], 2 + 4 * kWGroups);   // MMA, LSE and summing warps
        }
        mbar_init(&sm.drain, 1);
        sm.abort = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    // the LSE k-step: ones against a row's three parts, zeros behind them
    for (int i = threadIdx.x; i < kWBufs * kWCols + kWTile; i += kWThreads) {
        uint8_t *row = i < kWBufs * kWCols ? kw_row_x(sm.qx[i / kWCols], i % kWCols)
                                           : kw_row_x(sm.kx, i - kWBufs * kWCols);
        *reinterpret_cast<uint4 *>(row) =
            i < kWBufs * kWCols ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(0x3f803f80u, 0x3f80u, 0u, 0u);
        *reinterpret_cast<uint4 *>(row + 128) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
    if (warp == 1) {
        tmem_alloc(&sm.tmem_base, kWTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    griddep_wait();
    if (warp == 0)
        kw_producer<MANY>(&tm_k, tm_q, a, sm, lane);
    else if (warp == 1)
        kw_mma<MANY>(a, sm, tmem, lane);
    else if (warp == 2)
        kw_lse<MANY>(a, sm, lane);
    else if (warp == 3 && a.one_each && blockIdx.x == 0)
        kw_check(a, lane, 32);
    else if (warp >= kWFirstWarp)
        kw_sum(a, sm, tmem, warp, lane);
    __syncwarp();
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
    griddep_wait();
    const int64_t at = static_cast<int64_t>(u) * a.Lmax + j;
    const int64_t step = static_cast<int64_t>(a.B) * a.Hkv * a.Lmax;
    float w = 0.f;
#pragma unroll 4
    for (int p = 0; p < a.parts; ++p)
        w += a.partial[p * step + at];
    a.weights[at] = a.accumulate ? a.weights[at] + w : w;
}

// How the work is cut, from the sizes alone and for this GPU's 152 SMs, so that a
// workspace and the result do not depend on where they are made.
//   many   more query columns than one tile holds: query tiles stream
//   parts  shares of a pair's queries: enough items for about four per SM, none
//          shorter than a tile's rows
//   run    pairs per item: one, except where one query tile serves all of them,
//          which costs about as much to load as they do: one item per SM, of at
//          most 8 pairs (17 GFLOP over 32K keys: 1 pair an item 67 us, 4 51)
struct KwPlan {
    bool many;
    int seg, parts, run;
    int64_t units;         // pairs of one sequence
};

static KwPlan kw_plan(int B, int Tq, int Lmax, int Hkv, int g)
{
    KwPlan p;
    p.seg = g == 1 ? kWCols : kWTile;
    p.many = ceil_div(Tq, 16) * 16 * g > kWCols;
    p.units = ceil_div(Lmax, kWKeys);
    const int64_t tiles = p.units * B * Hkv;
    const int64_t want = ceil_div(4 * 152, tiles), most = ceil_div(Tq, p.seg);
    const int64_t parts = want < most ? want : most;
    p.parts = static_cast<int>(parts < 1 ? 1 : parts > kWMaxParts ? kWMaxParts : parts);
    const int64_t run = p.many ? 1 : ceil_div(tiles, 152);
    p.run = static_cast<int>(run > 8 ? 8 : run);
    return p;
}

// A kernel whose prologue may run under the end of the call's one before it, if
// there is one.
template <typename... A>
static cudaError_t launch_kw_after(void (*kernel)(A...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                                   bool follows, const A &...args)
{
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = follows ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <bool MANY>
static cudaError_t launch_kw(const CUtensorMap &tk, const KwMaps &tq, const KwArgs &a, int sms, int dev, cudaStream_t st)
{
    static bool attr_done[64] = {};   // the attribute is set once per device
    if (dev >= 64 || !attr_done[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(key_weights_kernel<MANY>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(kKwSmemBytes));
        if (e != cudaSuccess)
            return e;
        if (dev < 64)
            attr_done[dev] = true;
    }
    return launch_kw_after(key_weights_kernel<MANY>, dim3(static_cast<unsigned>(a.n_items < sms ? a.n_items : sms)),
                           kWThreads, kKwSmemBytes, st, !a.one_each, tk, tq, a);
}

} // namespace ea

using namespace ea;

extern "C" size_t ea_key_weights_workspace_size(int B, int Tq, int Lmax, int Hq, int Hkv, int d)
{
    if (B < 1 || Tq < 1 || Lmax < 1 || Lmax > EA_MAX_SEQ || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 ||
        d != EA_HEAD_DIM)
        return 0;
    const int parts = kw_plan(B, Tq, Lmax, Hkv, Hq / Hkv).parts;
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
    a.window = window < 2 * EA_MAX_SEQ ? window : 2 * EA_MAX_SEQ;   // (sums of positions stay in 32 bits)
    const KwPlan plan = kw_plan(B, Tq, Lmax, Hkv, a.g);
    a.parts = plan.parts;
    a.run = plan.run;
    a.seg = plan.seg;
    a.seg_log2 = plan.seg == kWTile ? 7 : 8;
    a.accumulate = accumulate != 0;
    a.c2 = scale * 1.4426950408889634f;
    a.inv_scale = 1.f / scale;
    const int64_t items = ceil_div(plan.units, a.run) * a.parts * B * Hkv;
    if (items >= (int64_t(1) << 31) - 1024)
        return EA_ERR_UNSUPPORTED;
    a.n_items = static_cast<int>(items);

    alignas(64) CUtensorMap tk;
    alignas(64) KwMaps tq;
    a.box = static_cast<int>(ceil_div(Tq, 16) * 16 < kWTile ? ceil_div(Tq, 16) * 16 : kWTile);
    if (!encode_tmap_bf16_4d(&tk, K, d, Hkv, Lmax, B, k_str, 64, kWTile, true) ||
        !encode_tmap_bf16_4d(&tq.rows, Q, d, Hq, Tq, B, q_str, 64, a.box, true) ||
        !encode_tmap_bf16_4d(&tq.r16, Q, d, Hq, Tq, B, q_str, 64, 16, true))
        return EA_ERR_INVALID_ARG;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return EA_ERR_CUDA;
    const int sms = num_sms(dev);
    if (sms <= 0)
        return EA_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    a.one_each = items <= sms;
    if (!a.one_each)
        kw_setup_kernel<<<1, 256, 0, st>>>(a);
    if ((plan.many ? launch_kw<true>(tk, tq, a, sms, dev, st)
                   : launch_kw<false>(tk, tq, a, sms, dev, st)) != cudaSuccess)
        return EA_ERR_CUDA;
    if (a.parts > 1 &&
        launch_kw_after(kw_join_kernel, dim3(static_cast<unsigned>(ceil_div(Lmax, 256)), static_cast<unsigned>(B * Hkv)),
                        256, 0, st, true, a) != cudaSuccess)
        return EA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? EA_OK : EA_ERR_CUDA;
}
