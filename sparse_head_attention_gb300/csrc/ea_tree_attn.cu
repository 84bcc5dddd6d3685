// ea_tree_attn.cu - attention of a tree of drafted tokens over a KV cache (bf16 or 8-bit,
// contiguous or paged; FA, SSA and block-sparse heads) and over the tree itself.
//
// The T nodes of a sequence times the g query heads of a KV head are the rows of a
// tcgen05 tile (128 TMEM lanes, a row a thread), 128 keys its columns:
//   S = Q K^T,  p = 2^(scale log2(e) S - m),  O += P V,  l += sum p
// with a running maximum m that the sums follow once it has grown by 2^8.  Keys come in
// tiles aligned to 128: the cache's, then one of the tree's own keys, whose mask is the
// node's ancestors.  Any other mask (lengths, windows, block rows) is 128 bits of a row
// and a tile; tiles that every row keeps whole carry none.
//
// What bounds it: each kept key's K and V are read once for up to 256 rows (two M tiles
// share a key tile), 64 KB a tile of bf16, which an SM receives in 1.45 us at the measured
// HBM rate; two M tiles take 0.55 us of tensor core and 0.5 of the SFU.  So HBM, up to
// some 500 rows a KV head.
//
// Work.  Key tiles of all (sequence, KV head, pair of M tiles) form one line, which is cut
// into equal ranges, one a CTA: no CTA idles, and at most two ranges of a CTA's begin or
// end inside a unit, so partial results are bounded by the grid, whatever the batch.  Every
// CTA finds its range itself (a scan over the units' tile counts).
//
// Roles of a CTA:
//   warps 0-7    two softmax warpgroups.  With two M tiles each has one; with one they take
//                key tiles in turn, each with its own O, m and l, joined at the range's end.
//   warp 8       ranges, Q, and by TMA the K and V tiles into a ring of 32 KB entries
//   warp 9       the MMAs, whichever product is ready first: S up to two tiles ahead
//   warps 10-11  V's rows that no query row keeps are zeroed before the product (0 * NaN is
//                NaN), and tiles of which some rows keep a key and others do not are searched
//                for infinities and NaN; such a tile's product is taken by the softmax warps,
//                key by key
//   warps 12-19  8-bit caches: codes from HBM to registers, times their scale (exact in bf16),
//                into the ring
#include <cuda.h>
#include <cuda_runtime.h>

#include "ea_cache.cuh"
#include "ea_internal.h"

namespace ea {

constexpr int kTTile = 128;
constexpr int kTBytes = kTTile * EA_HEAD_DIM * 2;     // a tile of K, V or Q: 32 KB
constexpr int kTHalf = kTBytes / 2;                   // 64 dims of 128 rows
constexpr int kTStages = 5;
constexpr int kTInfos = 16;                           // tile descriptions in flight: the ring holds three tiles
constexpr int kTReady = 8;
constexpr int kTSegs = 4;
constexpr int kTProducerWarp = 8, kTMmaWarp = 9, kTFixWarp = 10, kTFixWarps = 2, kTConvWarp = 12, kTConvWarps = 8;
constexpr int kTThreads = kTConvWarp * 32, kTThreadsQ8 = (kTConvWarp + kTConvWarps) * 32;
constexpr uint32_t kTColO = 256;                      // TMEM: S0, S1, O0, O1
constexpr uint32_t kTIdescQK = idesc_bf16_f32(128, 128, false, false);
constexpr uint32_t kTIdescPV = idesc_bf16_f32(128, 128, false, true);
constexpr float kTGrow = 8.f;                         // the maximum is followed once it grew by 2^8: p <= 2^8
constexpr int kTSms = 152;                            // a workspace's size depends on the grid

enum { kEdge = 1, kDraft = 2, kRow0 = 4, kRow1 = 8, kMixed = 16 };

struct TreeArgs {
    __nv_bfloat16 *O;
    int64_t o_sb, o_st, o_sh;
    float *LSE;
    const int32_t *seqlens, *n_nodes, *depth;
    const uint4 *mask;
    const uint8_t *m, *block_mask;
    int32_t *blk_count;
    uint32_t *blk_list;                  // key block | rows that keep it << 30
    int32_t *first, *last;               // CTAs of each (unit, pair of M tiles)
    float *part_o, *part_lse;            // [2 * grid][rows_slot][128], [2 * grid][rows_slot]
    ea_ws_header *hdr;
    CacheDev c;
    int B, T, Hq, Hkv, g, tpt, pairs, nBm, sink, window, min_tiles, box128, rows_slot;
    float scale_log2, grow;
};

struct TreeMaps {
    CUtensorMap q, kd, vd, k, v;
};

// One (sequence, KV head).
struct TreeUnit {
    int L, n, mode, nt, pairs;           // key tiles (the tree's included), pairs of M tiles
    int TA, TB, n0;                      // SSA: tiles [0, TA) and from TB on; keys below n0 are kept by all
    int need;                            // BLOCK: the block rows that the nodes lie in
    bool bad, dead;                      // reported; no key is kept
};

__device__ __forceinline__ TreeUnit tree_unit(const TreeArgs &a, int u)
{
    TreeUnit x;
    const int b = u / a.Hkv;
    x.n = a.n_nodes ? a.n_nodes[b] : a.T;
    x.L = a.seqlens[b];
    x.mode = a.m[u];
    x.bad = x.dead = false;
    if (x.n < 0 || x.n > a.T) {
        x.bad = true;
        x.n = 0;
    }
    if (x.L < 0 || x.L > a.c.cap || x.mode > EA_BLOCK ||
        (x.mode == EA_BLOCK && (!a.block_mask || (x.n > 0 && (static_cast<int64_t>(x.L) + x.n - 1) / EA_TILE >= a.nBm)))) {
        x.bad = x.dead = true;
        x.L = 0;
        x.mode = EA_FULL;
    }
    const int all = (x.L + kTTile - 1) / kTTile;
    x.TA = all;
    x.TB = all;
    x.n0 = x.L;
    x.need = 0;
    int tiles = all;
    if (x.mode == EA_SSA) {
        x.n0 = min(a.sink, x.L);
        x.TA = (x.n0 + kTTile - 1) / kTTile;
        // the window of depth 0, the longest
        x.TB = max(max(x.L - a.window + 1, 0) / kTTile, x.TA);
        tiles = x.TA + max(all - x.TB, 0);
    } else if (x.mode == EA_BLOCK) {
        tiles = a.blk_count[u];
        x.need = (x.L + x.n - 1) / EA_TILE > x.L / EA_TILE ? kRow0 | kRow1 : kRow0;
    }
    x.nt = tiles + 1;
    x.pairs = x.n > 0 ? ((x.n + a.tpt - 1) / a.tpt + 1) / 2 : 0;
    return x;
}

// A range's part of one unit.
struct TreeSeg {
    int valid;
    int b, h, v;                         // v: unit * pairs + pair
    int mode, L, n, dead;
    int tok0, two;                       // first node, and whether there are two M tiles
    int t0, t1, nt;                      // tiles [t0, t1) of nt
    int slot;                            // of the partial result
};

struct TreeTile {
    int key0, flags;
};

__device__ __forceinline__ TreeTile tree_tile(const TreeArgs &a, const TreeUnit &x, int u, int t)
{
    TreeTile r;
    if (t >= x.nt - 1) {
        r.key0 = x.L;
        r.flags = kEdge | kDraft | kMixed;
        return r;
    }
    r.flags = 0;
    if (x.mode == EA_BLOCK) {
        const int64_t at = static_cast<int64_t>(u) * a.nBm + t;
        const uint32_t e = in_bounds(t, a.nBm, &a.hdr->error) ? a.blk_list[at] : 0u;
        r.key0 = static_cast<int>(e & 0x3fffffffu) * kTTile;
        r.flags = static_cast<int>(e >> 30) * kRow0;
        if (r.flags != x.need)
            r.flags |= kEdge | kMixed;
    } else {
        r.key0 = (t < x.TA ? t : x.TB + t - x.TA) * kTTile;
        // kept by every row: below the sink's end, or in the window of the deepest node
        if (x.mode == EA_SSA && r.key0 + kTTile > x.n0 && r.key0 < x.L + x.n - a.window)
            r.flags |= kEdge | kMixed;
    }
    if (r.key0 + kTTile > x.L)
        r.flags |= kEdge;
    return r;
}

struct __align__(1024) TreeSmem {
    uint8_t q[2][kTBytes];
    uint8_t ring[kTStages][kTBytes];
    float2 ml[2][kTTile];                // a warpgroup's maximum and sum of each row; before: the scan
    uint64_t full[kTStages], empty[kTStages];
    uint64_t ready[kTReady];             // V has been looked over
    uint64_t seg_full[kTSegs], seg_empty[kTSegs];
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_full[2], o_done[2];
    uint64_t seg_done, ml_full, o_free, drain;
    TreeSeg seg[kTSegs];
    TreeTile tile[kTInfos];
    int odd[kTReady][kTFixWarps];        // V holds an infinity or a NaN
    int64_t count, off;                  // this CTA's range: tiles, and its start in the first unit
    int unit;
    uint32_t tmem_base;
    int abort;
};
constexpr size_t kTSmemBytes = sizeof(TreeSmem);
static_assert(kTSmemBytes <= 232448, "shared memory of one CTA");

__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(smem_u32(bar)), "r"(parity)
                 : "memory");
    return ok != 0;
}

// D[tmem] (+)= A[tmem] * B[smem].
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
                 : "memory");
}

__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr)
{
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr) : "memory");
    return r;
}

__device__ __forceinline__ float tree_lg2(float x)
{
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Columns below `n` of the 32 from 32 c on.
__device__ __forceinline__ uint32_t cols_below(int n, int c)
{
    const int k = n - 32 * c;
    return k <= 0 ? 0u : k >= 32 ? 0xffffffffu : (1u << k) - 1u;
}

// Segment number `it` (slot it % kTSegs), by a whole warp; false: gave up.
__device__ __forceinline__ bool tree_take(const TreeArgs &a, TreeSmem &sm, uint32_t it, TreeSeg &s)
{
    const int slot = it % kTSegs;
    if (!mbar_wait_warp(&sm.seg_full[slot], (it / kTSegs) & 1, &sm.abort, &a.hdr->error))
        return false;
    s = sm.seg[slot];
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(&sm.seg_empty[slot]);
    return s.valid != 0;
}

// ------------------------------------------------------------ ranges, Q, K and V
// Where 64 keys of a tile lie in the cache; row < 0: behind the sequence (not read).
__device__ __forceinline__ void tree_place(const TreeArgs &a, int b, int L, int key, int &outer, int &row)
{
    outer = b;
    row = key < L ? key : -1;
    if (row >= 0 && a.c.table) {
        const int pg = key / a.c.rows;
        row = key - pg * a.c.rows;
        outer = a.c.table[b * a.c.bt_stride + pg];
        if (outer < 0 || outer >= a.c.outer) {         // reported; reads zeros
            raise_error(&a.hdr->error, EA_DEVERR_CHECK);
            outer = -1;
        }
    }
}

template <bool Q8>
__device__ __forceinline__ void tree_producer(const TreeMaps &tm, const TreeArgs &a, TreeSmem &sm, int lane)
{
    uint32_t *err = &a.hdr->error;
    int u = sm.unit;
    int64_t off = sm.off, left = sm.count;
    uint32_t it = 0, entry = 0, tile = 0;
    bool ok = true;
    const uint32_t qbytes = static_cast<uint32_t>(a.g * a.tpt) * 256u;
    auto publish = [&](const TreeSeg &s) {
        const int slot = it % kTSegs;
        if (!mbar_wait_warp(&sm.seg_empty[slot], ((it / kTSegs) & 1) ^ 1, &sm.abort, err))
            return false;
        if (lane == 0) {
            sm.seg[slot] = s;
            mbar_arrive(&sm.seg_full[slot]);
        }
        __syncwarp();
        return true;
    };
    while (ok && left > 0) {
        const TreeUnit x = tree_unit(a, u);
        if (off >= static_cast<int64_t>(x.nt) * x.pairs) {
            ++u;
            off = 0;
            continue;
        }
        TreeSeg s;
        const int pair = static_cast<int>(off) / x.nt;
        s.valid = 1;
        s.b = u / a.Hkv;
        s.h = u % a.Hkv;
        s.v = u * a.pairs + pair;
        s.mode = x.mode;
        s.L = x.L;
        s.n = x.n;
        s.dead = x.dead;
        s.tok0 = 2 * pair * a.tpt;
        s.two = s.tok0 + a.tpt < x.n;
        s.t0 = static_cast<int>(off) - pair * x.nt;
        s.t1 = left < x.nt - s.t0 ? s.t0 + static_cast<int>(left) : x.nt;
        s.nt = x.nt;
        // a range holds one part that continues a unit (its first) and one that is continued at most
        s.slot = 2 * blockIdx.x + (s.t0 == 0 ? 1 : 0);
        off += s.t1 - s.t0;
        left -= s.t1 - s.t0;
        if (!publish(s))
            break;
        if (lane == 0) {
            if (s.t0 == 0)
                a.first[s.v] = blockIdx.x;
            if (s.t1 == s.nt)
                a.last[s.v] = blockIdx.x;
        }
        if (!mbar_wait_warp(&sm.q_empty, (it & 1) ^ 1, &sm.abort, err))
            break;
        if (lane == 0) {
            mbar_arrive_expect_tx(&sm.q_full, s.two ? 2 * qbytes : qbytes);
            for (int w = 0; w <= s.two; ++w)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
                    tma_load_4d(sm.q[w] + hf * kTHalf, &tm.q, 64 * hf, s.h * a.g, s.tok0 + w * a.tpt, s.b, &sm.q_full);
        }
        __syncwarp();
        ++it;
        // Lanes 2 i and 2 i + 1 hold the places of the halves of tile i of sixteen.
        TreeTile mine{};
        int row = -1, outer = 0;
        for (int t = s.t0; t < s.t1; ++t) {
            const int i = (t - s.t0) & 15;
            if (i == 0) {
                const int tt = t + (lane >> 1);
                if (tt < s.t1) {
                    mine = tree_tile(a, x, u, tt);
                    if (!Q8 && !(mine.flags & kDraft))
                        tree_place(a, s.b, s.L, mine.key0 + 64 * (lane & 1), outer, row);
                }
            }
            TreeTile ti;
            ti.key0 = __shfl_sync(0xffffffffu, mine.key0, 2 * i);
            ti.flags = __shfl_sync(0xffffffffu, mine.flags, 2 * i);
            int rw[2], ou[2];
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                rw[hf] = __shfl_sync(0xffffffffu, row, 2 * i + hf);
                ou[hf] = __shfl_sync(0xffffffffu, outer, 2 * i + hf);
            }
#pragma unroll
            for (int kv = 0; kv < 2; ++kv, ++entry) {
                const int st = entry % kTStages;
                if (!mbar_wait_warp(&sm.empty[st], ((entry / kTStages) & 1) ^ 1, &sm.abort, err)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    uint8_t *dst = sm.ring[st];
                    uint64_t *bar = &sm.full[st];
                    if (kv == 0)
                        sm.tile[tile % kTInfos] = ti;
                    if (ti.flags & kDraft) {
                        mbar_arrive_expect_tx(bar, kTBytes);
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf)
                            tma_load_4d(dst + hf * kTHalf, kv ? &tm.vd : &tm.kd, 64 * hf, s.h, 0, s.b, bar);
                    } else if (Q8) {
                        mbar_arrive(bar);
                    } else if (a.box128) {
                        mbar_arrive_expect_tx(bar, kTBytes);
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf)
                            tma_load_4d(dst + hf * kTHalf, kv ? &tm.v : &tm.k, 64 * hf, s.h, rw[0], ou[0], bar);
                    } else {
                        mbar_arrive_expect_tx(bar, rw[1] >= 0 ? kTBytes : kTHalf);
#pragma unroll
                        for (int p = 0; p < 2; ++p)
                            if (rw[p] >= 0)
#pragma unroll
                                for (int hf = 0; hf < 2; ++hf)
                                    tma_load_4d(dst + hf * kTHalf + p * (kTHalf / 2), kv ? &tm.v : &tm.k, 64 * hf, s.h,
                                                rw[p], ou[p], bar);
                    }
                }
                __syncwarp();
            }
            if (!ok)
                break;
            ++tile;
        }
    }
    TreeSeg none{};
    if (ok)
        publish(none);
    // Before leaving on an abort, let the copies already issued land.
    if (__any_sync(0xffffffffu, *static_cast<volatile int *>(&sm.abort))) {
        volatile int no_abort = 0;
        for (uint32_t n = entry > kTStages ? entry - kTStages : 0; n < entry; ++n)
            mbar_wait_warp(&sm.full[n % kTStages], (n / kTStages) & 1, &no_abort, nullptr);
        if (it > 0)
            mbar_wait_warp(&sm.q_full, (it - 1) & 1, &no_abort, nullptr);
    }
}

// ------------------------------------------------------------ products
// One thread.  Takes whichever is ready: the next S = Q K^T (at most two ahead of the
// products that have consumed theirs), or the next O += P V.
__device__ __forceinline__ void tree_mma(const TreeArgs &a, TreeSmem &sm, uint32_t tmem)
{
    volatile int *abort = &sm.abort;
    uint32_t *err = &a.hdr->error;
    uint32_t it = 0, tile0 = 0, p_cnt[2] = {0, 0};
    bool ok = true;
    for (; ok; ++it) {
        const int slot = it % kTSegs;
        if (!mbar_wait(&sm.seg_full[slot], (it / kTSegs) & 1, abort, err))
            break;
        const int valid = sm.seg[slot].valid, two = sm.seg[slot].two, nt = sm.seg[slot].t1 - sm.seg[slot].t0;
        mbar_arrive(&sm.seg_empty[slot]);
        if (!valid)
            break;
        if (!mbar_wait(&sm.q_full, it & 1, abort, err))
            break;
        const int N = nt << two;
        int qk = 0, pv = 0;
        bool o_free = it == 0;
        uint64_t t0 = 0;
        while (pv < N) {
            bool did = false;
            if (qk < N && qk < pv + 2) {
                const int t = qk >> two, w = qk & 1;
                const uint32_t e = 2 * (tile0 + t);
                const int st = e % kTStages;
                if (mbar_test(&sm.full[st], (e / kTStages) & 1)) {
                    tc_fence_after();
                    const uint32_t qa = smem_u32(sm.q[two ? w : 0]), ka = smem_u32(sm.ring[st]);
#pragma unroll
                    for (int k = 0; k < EA_HEAD_DIM / 16; ++k) {
                        const uint32_t o = (k >> 2) * kTHalf + (k & 3) * 32;
                        tc_mma(tmem + 128 * w, sdesc_sw128(qa + o, 16, 1024), sdesc_sw128(ka + o, 16, 1024), kTIdescQK, k > 0);
                    }
                    tc_commit(&sm.s_full[w]);
                    if (!two || w == 1)
                        tc_commit(&sm.empty[st]);
                    if (++qk == N)
                        tc_commit(&sm.q_empty);
                    did = true;
                }
            }
            if (pv < qk) {
                const int t = pv >> two, w = pv & 1;
                const uint32_t tile = tile0 + t, e = 2 * tile + 1;
                const int st = e % kTStages;
                if (!o_free)
                    o_free = mbar_test(&sm.o_free, (it - 1) & 1);
                if (o_free && mbar_test(&sm.p_full[w], p_cnt[w] & 1) && mbar_test(&sm.ready[tile % kTReady], (tile / kTReady) & 1)) {
                    tc_fence_after();
                    const int *odd = sm.odd[tile % kTReady];
                    if (!(odd[0] | odd[1])) {
                        const uint32_t va = smem_u32(sm.ring[st]);
                        // (a warpgroup's first product of the range overwrites what its O held)
                        const bool first = pv < 2;
#pragma unroll
                        for (int k = 0; k < kTTile / 16; ++k)
                            tc_mma_ts(tmem + kTColO + 128 * w, tmem + 128 * w + 8 * k, sdesc_sw128(va + k * 2048, kTHalf, 1024),
                                      kTIdescPV, !first || k > 0);
                    }
                    tc_commit(&sm.o_done[w]);
                    if (!two || w == 1)
                        tc_commit(&sm.empty[st]);
                    ++p_cnt[w];
                    if (++pv == N)
                        tc_commit(&sm.seg_done);
                    did = true;
                }
            }
            if (did) {
                t0 = 0;
                continue;
            }
            if (*abort) {
                ok = false;
                break;
            }
            const uint64_t now = globaltimer_ns();
            if (t0 == 0) {
                t0 = now;
            } else if (now - t0 > EA_WAIT_TIMEOUT_NS) {
                raise_error(err, EA_DEVERR_TIMEOUT);
                *abort = 1;
                ok = false;
                break;
            }
        }
        tile0 += nt;
    }
    // All of this thread's MMAs must have completed before TMEM is released.
    tc_commit(&sm.drain);
    volatile int no_abort = 0;
    mbar_wait(&sm.drain, 0, &no_abort, err);
}

// ------------------------------------------------------------ V's rows
__device__ __forceinline__ uint32_t odd_bf16x2(uint32_t w)
{
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

__device__ __forceinline__ void tree_fix(const TreeArgs &a, TreeSmem &sm, int warp, int lane)
{
    uint32_t *err = &a.hdr->error;
    uint32_t tile = 0;
    TreeSeg s;
    for (uint32_t it = 0; tree_take(a, sm, it, s); ++it)
        for (int t = s.t0; t < s.t1; ++t, ++tile) {
            const uint32_t e = 2 * tile;
            const int ks = e % kTStages, vs = (e + 1) % kTStages;
            if (!mbar_wait_warp(&sm.full[ks], (e / kTStages) & 1, &sm.abort, err))
                return;
            const TreeTile ti = sm.tile[tile % kTInfos];
            if (!mbar_wait_warp(&sm.full[vs], ((e + 1) / kTStages) & 1, &sm.abort, err))
                return;
            bool odd = false;
            if (ti.flags & kEdge) {
                const int nv = (ti.flags & kDraft) ? s.n : min(kTTile, s.L - ti.key0);
                const int from = (ti.flags & kMixed) ? 0 : nv * 16;
                // 16 bytes of row i / 16: eight of each half (their order in a row does not matter)
#pragma unroll 4
                for (int i = from + (warp - kTFixWarp) * 32 + lane; i < kTTile * 16; i += kTFixWarps * 32) {
                    uint4 *p = reinterpret_cast<uint4 *>(sm.ring[vs] + ((i >> 3) & 1) * kTHalf + (i >> 4) * 128 + (i & 7) * 16);
                    if ((i >> 4) >= nv) {
                        *p = make_uint4(0u, 0u, 0u, 0u);
                    } else {
                        const uint4 v = *p;
                        odd |= odd_bf16x2(v.x) | odd_bf16x2(v.y) | odd_bf16x2(v.z) | odd_bf16x2(v.w);
                    }
                }
                fence_proxy_async_smem();
            }
            odd = __any_sync(0xffffffffu, odd);
            if (lane == 0) {
                sm.odd[tile % kTReady][warp - kTFixWarp] = odd;
                mbar_arrive(&sm.ready[tile % kTReady]);
                mbar_arrive(&sm.empty[ks]);
                mbar_arrive(&sm.empty[vs]);
            }
            __syncwarp();
        }
}

// ------------------------------------------------------------ 8-bit caches
// 16 codes of one row, times its scale, as bf16 (exact: at most 8 bits).
template <bool E4M3>
__device__ __forceinline__ void put16(uint8_t *tile, int row, int chunk, const uint4 &c, float s)
{
    uint32_t o[8];
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h[2];
        codes_f16<E4M3>(w[i], h[0], h[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float2 v = f16_f32(h[k]);
            o[2 * i + k] = pack_bf16x2(v.x * s, v.y * s);
        }
    }
    // 32 bytes at column 32 (chunk % 4) of the row's half, 16-byte pieces swizzled; the two
    // halves' lanes store their pieces in opposite order, so that they meet other banks
    uint8_t *p = tile + (chunk >> 2) * kTHalf + row * 128;
    const int c0 = (chunk & 3) * 2, flip = chunk >> 2;
    const uint4 a0 = make_uint4(o[0], o[1], o[2], o[3]), a1 = make_uint4(o[4], o[5], o[6], o[7]);
    *reinterpret_cast<uint4 *>(p + (((c0 + flip) ^ (row & 7)) << 4)) = flip ? a1 : a0;
    *reinterpret_cast<uint4 *>(p + (((c0 + 1 - flip) ^ (row & 7)) << 4)) = flip ? a0 : a1;
}

template <bool E4M3>
__device__ __forceinline__ void tree_convert(const TreeArgs &a, TreeSmem &sm, int ct, int lane)
{
    uint32_t *err = &a.hdr->error;
    uint32_t entry = 0;
    TreeSeg s;
    const int chunk = ct & 7, r0 = ct >> 3;
    for (uint32_t it = 0; tree_take(a, sm, it, s); ++it) {
        const int u = s.b * a.Hkv + s.h;
        const TreeUnit x = tree_unit(a, u);
        struct Codes {
            uint4 c[2][4];
            float f[2][4];
        };
        auto load = [&](int t, Codes &z) {
            const TreeTile ti = t < s.t1 ? tree_tile(a, x, u, t) : TreeTile{0, kDraft};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = ti.key0 + 32 * i + r0;
                int outer = 0, row = -1;
                if (!(ti.flags & kDraft))
                    tree_place(a, s.b, s.L, key, outer, row);
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    z.c[kv][i] = make_uint4(0u, 0u, 0u, 0u);
                    z.f[kv][i] = 0.f;
                    if (row >= 0 && outer >= 0) {
                        z.c[kv][i] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.c.code[kv]) +
                                                                           outer * a.c.s_outer + row * a.c.s_row +
                                                                           s.h * a.c.s_head + 16 * chunk));
                        z.f[kv][i] = __ldg(a.c.scale[kv] + (static_cast<int64_t>(outer) * a.c.Hkv + s.h) * a.c.nsb +
                                           (row >> a.c.log2sb));
                    }
                }
            }
        };
        auto put = [&](int t, const Codes &z) {
            const bool draft = t == s.nt - 1;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv, ++entry) {
                const int st = entry % kTStages;
                if (!mbar_wait_warp(&sm.empty[st], ((entry / kTStages) & 1) ^ 1, &sm.abort, err))
                    return false;
                if (!draft) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        put16<E4M3>(sm.ring[st], 32 * i + r0, chunk, z.c[kv][i], z.f[kv][i]);
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sm.full[st]);
            }
            return true;
        };
        Codes z0;
        for (int t = s.t0; t < s.t1; ++t) {
            load(t, z0);
            if (!put(t, z0))
                return;
        }
    }
}

// ------------------------------------------------------------ softmax
__device__ __forceinline__ void tree_softmax(const TreeArgs &a, TreeSmem &sm, uint32_t tmem, int warp, int lane)
{
    const float NEG_INF = -__int_as_float(0x7f800000);
    uint32_t *err = &a.hdr->error;
    const int wg = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_base + 128 * wg, to = tmem + lane_base + kTColO;
    uint32_t own = 0, tile0 = 0, joined = 0;
    TreeSeg s;
    for (uint32_t it = 0; tree_take(a, sm, it, s); ++it) {
        const int mt = s.two ? wg : 0, tl = r / a.g, hh = r - tl * a.g;
        const int t = s.tok0 + mt * a.tpt + tl;
        const bool valid = tl < a.tpt && t < s.n;
        const bool active = __any_sync(0xffffffffu, valid);
        const int64_t node = static_cast<int64_t>(s.b) * a.T + t;
        int d = 0;
        if (valid) {
            d = a.depth[node];
            if (d < 0 || d >= s.n) {
                raise_error(err, EA_DEVERR_CHECK);
                d = d < 0 ? 0 : s.n - 1;
            }
        }
        float m = NEG_INF, l = 0.f;
        int steps = 0;
        for (int tt = s.t0 + (s.two ? 0 : wg); tt < s.t1; tt += s.two ? 1 : 2, ++own, ++steps) {
            if (!mbar_wait_warp(&sm.s_full[wg], own & 1, &sm.abort, err))
                return;
            if (active) {
                if (own > 0 && !mbar_wait_warp(&sm.o_done[wg], (own - 1) & 1, &sm.abort, err))
                    return;
                tc_fence_after();
                const uint32_t tile = tile0 + (tt - s.t0);
                const TreeTile ti = sm.tile[tile % kTInfos];
                uint32_t keep[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
                bool odd = false;
                if (ti.flags & kEdge) {
                    if (ti.flags & kDraft) {
                        const uint4 up = valid && !s.dead ? a.mask[node] : make_uint4(0u, 0u, 0u, 0u);
                        const uint32_t w[4] = {up.x, up.y, up.z, up.w};
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            keep[c] = w[c] & cols_below(s.n, c);
                        // which ancestors the head's mode keeps at this node's position
                        const bool ssa = s.mode == EA_SSA && d >= a.window, blk = s.mode == EA_BLOCK;
                        if (ssa || blk) {
                            const int64_t mrow = (static_cast<int64_t>(s.b) * a.Hkv + s.h) * a.nBm + (s.L + d) / EA_TILE;
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                for (uint32_t left = keep[c]; left; left &= left - 1) {
                                    const int j = 32 * c + __ffs(left) - 1;
                                    const int dj = a.depth[static_cast<int64_t>(s.b) * a.T + j], pos = s.L + dj;
                                    bool in;
                                    if (ssa)
                                        in = pos < a.sink || d - dj < a.window;
                                    else
                                        in = dj >= 0 && pos / EA_TILE < a.nBm && a.block_mask[mrow * a.nBm + pos / EA_TILE] != 0;
                                    if (!in)
                                        keep[c] &= ~(left & (0u - left));
                                }
                        }
                    } else {
                        const int lim = s.L - ti.key0;
                        const bool row_in = s.mode != EA_BLOCK ||
                                            (ti.flags & ((s.L + d) / EA_TILE > s.L / EA_TILE ? kRow1 : kRow0));
                        const int sink = a.sink - ti.key0;                       // columns below are kept,
                        const int win = s.L - ti.key0 + d - a.window + 1;        // and those from here on
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            keep[c] = row_in ? cols_below(lim, c) : 0u;
                            if (s.mode == EA_SSA)
                                keep[c] &= cols_below(sink, c) | ~cols_below(win, c);
                        }
                    }
                    if (ti.flags & kMixed) {
                        if (!mbar_wait_warp(&sm.ready[tile % kTReady], (tile / kTReady) & 1, &sm.abort, err))
                            return;
                        odd = (sm.odd[tile % kTReady][0] | sm.odd[tile % kTReady][1]) != 0;
                    }
                }
                const bool edge = (ti.flags & kEdge) != 0;
                __syncwarp();
                float mx = NEG_INF;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t x[32];
                    tmem_ld32(ts + 32 * c, x);
                    tmem_wait_ld();
                    if (edge) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            x[i] = (keep[c] >> i) & 1u ? x[i] : 0xff800000u;
                    }
#pragma unroll
                    for (int i = 0; i < 32; i += 2)
                        mx = max3f(mx, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
                }
                const bool grew = mx > m + a.grow;
                if (__any_sync(0xffffffffu, grew)) {
                    const float f = grew && m != NEG_INF ? ex2((m - mx) * a.scale_log2) : 1.f;
                    m = grew ? mx : m;
                    l *= f;
                    if (steps > 0) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t x[32];
                            tmem_ld32(to + 128 * wg + 32 * c, x);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
                            tmem_st32(to + 128 * wg + 32 * c, x);
                        }
                        tmem_wait_st();
                    }
                }
                const float mb = m == NEG_INF ? 0.f : m * a.scale_log2;
                if (!odd) {
                    float sum[2] = {0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t x[32], p[16];
                        tmem_ld32(ts + 32 * c, x);
                        tmem_wait_ld();
                        if (edge) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                x[i] = (keep[c] >> i) & 1u ? x[i] : 0xff800000u;
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float p0 = ex2(fmaf(__uint_as_float(x[2 * i]), a.scale_log2, -mb));
                            const float p1 = ex2(fmaf(__uint_as_float(x[2 * i + 1]), a.scale_log2, -mb));
                            sum[0] += p0;
                            sum[1] += p1;
                            p[i] = pack_bf16x2(p0, p1);
                        }
                        tmem_st16(ts + 16 * c, p);
                    }
                    l += sum[0] + sum[1];
                } else {
                    // V holds infinities or NaN in a tile that rows keep differently: the kept keys
                    // one by one, so that none reaches a row that does not keep it (the first ones of
                    // a range write O, once nobody reads the last range's)
                    if (steps == 0 && it > 0 && !mbar_wait_warp(&sm.o_free, (it - 1) & 1, &sm.abort, err))
                        return;
                    float sum = 0.f;
                    for (int c = 0; c < 4; ++c) {
                        uint32_t o[32];
                        if (steps > 0) {
                            tmem_ld32(to + 128 * wg + 32 * c, o);
                            tmem_wait_ld();
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[i] = 0u;
                        }
                        const uint32_t e = 2 * tile + 1;
                        const uint8_t *half = sm.ring[e % kTStages] + (c >> 1) * kTHalf;
#pragma unroll
                        for (int kc = 0; kc < 4; ++kc)
                            for (int k = 0; k < 32; ++k) {
                                __syncwarp();
                                const uint32_t raw = tmem_ld1(ts + 32 * kc + k);
                                tmem_wait_ld();
                                if (!((keep[kc] >> k) & 1u))
                                    continue;                    // (lanes meet again above)
                                const float p = ex2(fmaf(__uint_as_float(raw), a.scale_log2, -mb));
                                sum += c == 0 ? p : 0.f;
                                const int row = 32 * kc + k;
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const uint4 v = *reinterpret_cast<const uint4 *>(
                                        half + row * 128 + ((((c & 1) * 4 + j) ^ (row & 7)) << 4));
                                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                    for (int q = 0; q < 4; ++q) {
                                        float *f = reinterpret_cast<float *>(o) + 8 * j + 2 * q;
                                        f[0] = fmaf(p, __uint_as_float(w[q] << 16), f[0]);
                                        f[1] = fmaf(p, __uint_as_float(w[q] & 0xffff0000u), f[1]);
                                    }
                                }
                            }
                        __syncwarp();
                        tmem_st32(to + 128 * wg + 32 * c, o);
                    }
                    l += sum;
                }
                tmem_wait_st();
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sm.p_full[wg]);
        }
        tile0 += s.t1 - s.t0;

        // the range's part of this unit is complete
        if (!mbar_wait_warp(&sm.seg_done, it & 1, &sm.abort, err))
            return;
        tc_fence_after();
        float f0 = 1.f, f1 = 0.f;
        bool both = false;
        float M = m == NEG_INF ? NEG_INF : m * a.scale_log2;
        if (!s.two) {
            sm.ml[wg][r] = make_float2(M, l);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sm.ml_full);
            if (!mbar_wait_warp(&sm.ml_full, joined++ & 1, &sm.abort, err))
                return;
            const float2 x0 = sm.ml[0][r], x1 = sm.ml[1][r];
            M = fmaxf(x0.x, x1.x);
            // 1 where nothing but NaN (or no key) was met, so that a NaN stays
            f0 = x0.x == NEG_INF ? 1.f : ex2(x0.x - M);
            f1 = x1.x == NEG_INF ? 1.f : ex2(x1.x - M);
            both = s.t1 - s.t0 > 1;
            l = both ? x0.y * f0 + x1.y * f1 : x0.y * f0;
        }
        if (active) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const bool whole = s.t0 == 0 && s.t1 == s.nt;
            const int64_t prow = static_cast<int64_t>(s.slot) * a.rows_slot + mt * kTTile + r;
            const int c0 = s.two ? 0 : 2 * wg, c1 = s.two ? 4 : c0 + 2;
            for (int c = c0; c < c1; ++c) {
                uint32_t x[32];
                __syncwarp();
                tmem_ld32(to + (s.two ? 128 * wg : 0) + 32 * c, x);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    x[i] = __float_as_uint(__uint_as_float(x[i]) * f0);
                if (both) {
                    uint32_t y[32];
                    tmem_ld32(to + 128 + 32 * c, y);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        x[i] = __float_as_uint(fmaf(__uint_as_float(y[i]), f1, __uint_as_float(x[i])));
                }
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    x[i] = l == 0.f ? 0u : __float_as_uint(__uint_as_float(x[i]) * inv);
                if (valid) {
                    if (whole) {
                        __nv_bfloat16 *o = a.O + s.b * a.o_sb + t * a.o_st + (s.h * a.g + hh) * a.o_sh + 32 * c;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t w[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                w[k] = pack_bf16x2(__uint_as_float(x[8 * i + 2 * k]), __uint_as_float(x[8 * i + 2 * k + 1]));
                            reinterpret_cast<uint4 *>(o)[i] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    } else if (in_bounds(prow, 2 * static_cast<int64_t>(gridDim.x) * a.rows_slot, err)) {
                        float *o = a.part_o + prow * EA_HEAD_DIM + 32 * c;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            st_global_v8(o + 8 * i, x + 8 * i);
                    }
                }
            }
            if (valid && (s.two || wg == 0)) {
                const float l2 = l == 0.f ? NEG_INF : (M == NEG_INF ? 0.f : M) + tree_lg2(l);
                if (!whole) {
                    if (in_bounds(prow, 2 * static_cast<int64_t>(gridDim.x) * a.rows_slot, err))
                        a.part_lse[prow] = l2;
                } else if (a.LSE) {
                    a.LSE[(static_cast<int64_t>(s.b) * a.Hq + s.h * a.g + hh) * a.T + t] = l2 * 0.69314718055994531f;
                }
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&sm.o_free);
    }
}

// ------------------------------------------------------------ kernels
// This CTA's range of the line of tiles: [i W / G, (i + 1) W / G) of its W tiles, G CTAs (fewer
// where a range would be shorter than min_tiles).
__device__ __forceinline__ void tree_range(const TreeArgs &a, TreeSmem &sm)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, units = a.B * a.Hkv;
    const int per = (units + blockDim.x - 1) / static_cast<int>(blockDim.x);
    const int lo = min(tid * per, units), hi = min(lo + per, units);
    int64_t mine = 0;
    bool bad = false;
    for (int u = lo; u < hi; ++u) {
        const TreeUnit x = tree_unit(a, u);
        mine += static_cast<int64_t>(x.nt) * x.pairs;
        bad |= x.bad;
    }
    if (bad && blockIdx.x == 0)
        raise_error(&a.hdr->error, EA_DEVERR_CHECK);
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += v;
    }
    int64_t *tot = reinterpret_cast<int64_t *>(sm.ml);
    if (lane == 31)
        tot[warp] = incl;
    if (tid == 0)
        sm.count = 0;
    __syncthreads();
    int64_t before = 0, W = 0;
    for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) {
        before += w < warp ? tot[w] : 0;
        W += tot[w];
    }
    int64_t base = before + incl - mine;
    const int64_t G = max(static_cast<int64_t>(1), min(static_cast<int64_t>(gridDim.x), W / a.min_tiles));
    const int64_t i = blockIdx.x;
    const int64_t start = i * W / G, end = (i + 1) * W / G;
    if (i < G && start < end && start >= base && start < base + mine)
        for (int u = lo; u < hi; ++u) {
            const TreeUnit x = tree_unit(a, u);
            const int64_t w = static_cast<int64_t>(x.nt) * x.pairs;
            if (start < base + w) {
                sm.unit = u;
                sm.off = start - base;
                sm.count = end - start;
                break;
            }
            base += w;
        }
    __syncthreads();
}

template <int FMT>
__global__ void __launch_bounds__(FMT == EA_CACHE_BF16 ? kTThreads : kTThreadsQ8, 1)
    tree_attn_kernel(const __grid_constant__ TreeMaps tm, const TreeArgs a)
{
    constexpr bool kQ8 = FMT != EA_CACHE_BF16;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    TreeSmem &sm = *reinterpret_cast<TreeSmem *>(smem_raw);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (smem_u32(smem_raw) & 1023u) {                  // the operands' layout needs it
        if (threadIdx.x == 0)
            raise_error(&a.hdr->error, EA_DEVERR_BOUNDS);
        return;
    }
    if (threadIdx.x == 0) {
        const int users = 1 + 8 + kTFixWarps + (kQ8 ? kTConvWarps : 0);
        for (int s = 0; s < kTStages; ++s) {
            mbar_init(&sm.full[s], 1 + (kQ8 ? kTConvWarps : 0));
            mbar_init(&sm.empty[s], 1 + kTFixWarps);
        }
        for (int s = 0; s < kTReady; ++s)
            mbar_init(&sm.ready[s], kTFixWarps);
        for (int s = 0; s < kTSegs; ++s) {
            mbar_init(&sm.seg_full[s], 1);
            mbar_init(&sm.seg_empty[s], users);
        }
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_empty, 1);
        for (int w = 0; w < 2; ++w) {
            mbar_init(&sm.s_full[w], 1);
            mbar_init(&sm.p_full[w], 4);
            mbar_init(&sm.o_done[w], 1);
        }
        mbar_init(&sm.seg_done, 1);
        mbar_init(&sm.ml_full, 8);
        mbar_init(&sm.o_free, 8);
        mbar_init(&sm.drain, 1);
        sm.abort = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == kTMmaWarp) {
        tmem_alloc(&sm.tmem_base, 512);
        tmem_relinquish();
    }
    if (warp == kTProducerWarp && lane == 0) {
        tma_prefetch_desc(&tm.q);
        tma_prefetch_desc(&tm.k);
        tma_prefetch_desc(&tm.v);
    }
    griddep_wait();
    griddep_launch_dependents();
    tree_range(a, sm);                                  // (its barriers order the set-up too)
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;

    if (warp < 8)
        tree_softmax(a, sm, tmem, warp, lane);
    else if (warp == kTProducerWarp)
        tree_producer<kQ8>(tm, a, sm, lane);
    else if (warp == kTMmaWarp) {
        if (lane == 0)
            tree_mma(a, sm, tmem);
    } else if (warp < kTConvWarp)
        tree_fix(a, sm, warp, lane);
    else if constexpr (kQ8)
        tree_convert<FMT == EA_CACHE_E4M3>(a, sm, threadIdx.x - kTConvWarp * 32, lane);

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kTMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// One CTA per unit: the key blocks below L that the block rows of the nodes' positions keep
// (L / 128 and, where the deepest node may reach it, the next), ascending.
constexpr int kTBlkThreads = 256;

__global__ void __launch_bounds__(kTBlkThreads) tree_blocks_kernel(const TreeArgs a)
{
    __shared__ int warp_tot[kTBlkThreads / 32];
    const int u = blockIdx.x, tid = threadIdx.x, lane = tid % 32, warp = tid / 32, b = u / a.Hkv;
    griddep_launch_dependents();
    const int L = a.seqlens[b], n = a.n_nodes ? a.n_nodes[b] : a.T;
    int count = 0;
    if (a.m[u] == EA_BLOCK && L > 0 && L <= a.c.cap && n > 0 && n <= a.T &&
        (static_cast<int64_t>(L) + n - 1) / EA_TILE < a.nBm) {
        const int r0 = L / EA_TILE, last = (L - 1) / EA_TILE;
        const bool two = (L + n - 1) / EA_TILE > r0;
        const uint8_t *row = a.block_mask + (static_cast<int64_t>(u) * a.nBm + r0) * a.nBm;
        uint32_t *list = a.blk_list + static_cast<int64_t>(u) * a.nBm;
        for (int k0 = 0; k0 <= last; k0 += kTBlkThreads) {
            const int kb = k0 + tid;
            uint32_t bits = 0;
            if (kb <= last) {
                bits = row[kb] != 0 ? 1u : 0u;
                if (two && row[a.nBm + kb] != 0)
                    bits |= 2u;
            }
            const uint32_t votes = __ballot_sync(0xffffffffu, bits != 0);
            if (lane == 0)
                warp_tot[warp] = __popc(votes);
            __syncthreads();
            int pos = count + __popc(votes & ((1u << lane) - 1u)), total = 0;
#pragma unroll
            for (int w = 0; w < kTBlkThreads / 32; ++w) {
                pos += w < warp ? warp_tot[w] : 0;
                total += warp_tot[w];
            }
            if (bits && in_bounds(pos, a.nBm, &a.hdr->error))
                list[pos] = static_cast<uint32_t>(kb) | bits << 30;
            count += total;
            __syncthreads();
        }
    }
    if (tid == 0)
        a.blk_count[u] = count;
}

// A warp per (sequence, node, query head) whose unit was cut: joins the parts by their
// weights 2^(lse - max), in the order of the keys.
constexpr int kTMergeWarps = 8;

__global__ void __launch_bounds__(kTMergeWarps * 32) tree_merge_kernel(const TreeArgs a)
{
    const float NEG_INF = -__int_as_float(0x7f800000);
    griddep_wait();
    const int lane = threadIdx.x % 32;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kTMergeWarps + threadIdx.x / 32;
    if (row >= static_cast<int64_t>(a.B) * a.T * a.Hq)
        return;
    const int qh = static_cast<int>(row % a.Hq), t = static_cast<int>(row / a.Hq % a.T), b = static_cast<int>(row / a.Hq / a.T);
    int n = a.n_nodes ? a.n_nodes[b] : a.T;
    if (n < 0 || n > a.T || t >= n)
        return;
    const int h = qh / a.g, hh = qh - h * a.g, mt = t / a.tpt;
    const int v = (b * a.Hkv + h) * a.pairs + mt / 2;
    const int c0 = a.first[v], c1 = a.last[v];
    if (c0 >= c1 || !in_bounds(c1, kTSms, &a.hdr->error) || !in_bounds(c0, kTSms, &a.hdr->error))
        return;                                          // written by its CTA
    const int64_t in_slot = (mt & 1) * kTTile + (t - mt * a.tpt) * a.g + hh;
    auto part = [&](int c) { return (2 * static_cast<int64_t>(c) + (c == c0 ? 1 : 0)) * a.rows_slot + in_slot; };
    float M = NEG_INF;
    for (int c = c0 + lane; c <= c1; c += 32)
        M = fmaxf(M, a.part_lse[part(c)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float ref = M == NEG_INF ? 0.f : M;
    float w = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int cb = c0; cb <= c1; cb += 32) {
        const float mine = cb + lane <= c1 ? ex2(a.part_lse[part(cb + lane)] - ref) : 0.f;
        const int k1 = min(32, c1 - cb + 1);
#pragma unroll 4
        for (int k = 0; k < k1; ++k) {
            const float e = __shfl_sync(0xffffffffu, mine, k);
            const float4 x = *reinterpret_cast<const float4 *>(a.part_o + part(cb + k) * EA_HEAD_DIM + 4 * lane);
            w += e;
            acc.x = fmaf(e, x.x, acc.x);
            acc.y = fmaf(e, x.y, acc.y);
            acc.z = fmaf(e, x.z, acc.z);
            acc.w = fmaf(e, x.w, acc.w);
        }
    }
    const float inv = w == 0.f ? 0.f : 1.f / w;
    const uint2 o = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    *reinterpret_cast<uint2 *>(a.O + b * a.o_sb + t * a.o_st + qh * a.o_sh + 4 * lane) = o;
    if (a.LSE && lane == 0)
        a.LSE[(static_cast<int64_t>(b) * a.Hq + qh) * a.T + t] =
            (w == 0.f ? NEG_INF : ref + tree_lg2(w)) * 0.69314718055994531f;
}

// ------------------------------------------------------------ host
constexpr int kTMinTiles = 2;

struct TreeWs {
    size_t first, last, blk_count, blk_list, part_lse, part_o, total;
    int tpt, pairs, rows_slot;
};

static TreeWs tree_ws_layout(int B, int T, int Hq, int Hkv, int Lmax)
{
    TreeWs w{};
    const int g = Hq / Hkv;
    w.tpt = kTTile / g;
    const int mtiles = static_cast<int>(ceil_div(T, w.tpt));
    w.pairs = (mtiles + 1) / 2;
    w.rows_slot = mtiles > 1 ? 2 * kTTile : kTTile;
    const size_t units = static_cast<size_t>(B) * Hkv;
    size_t off = sizeof(ea_ws_header);
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align_up(off + bytes, 256);
        return at;
    };
    w.first = take(sizeof(int32_t) * units * w.pairs);
    w.last = take(sizeof(int32_t) * units * w.pairs);
    w.blk_count = take(sizeof(int32_t) * units);
    w.blk_list = take(sizeof(uint32_t) * units * static_cast<size_t>(ceil_div(Lmax, EA_TILE)));
    w.part_lse = take(sizeof(float) * 2 * kTSms * w.rows_slot);
    w.part_o = take(sizeof(float) * 2 * kTSms * w.rows_slot * EA_HEAD_DIM);
    w.total = off;
    return w;
}

static bool tree_sizes_ok(int B, int T, int Hq, int Hkv, int d)
{
    return B >= 1 && T >= 1 && T <= EA_MAX_TREE && Hkv >= 1 && Hq >= 1 && Hq % Hkv == 0 && Hq / Hkv <= 64 &&
           d == EA_HEAD_DIM && B <= 65535 && Hkv <= 65535 && static_cast<int64_t>(B) * Hkv <= (int64_t(1) << 24) &&
           static_cast<int64_t>(B) * T * Hq <= (int64_t(1) << 33);
}

static bool tree_tensor(const void *p, const int64_t *str)
{
    if (!p || !str || str[3] != 1 || (reinterpret_cast<uintptr_t>(p) & 15u))
        return false;
    for (int k = 0; k < 3; ++k)
        if (str[k] <= 0 || str[k] % 8)
            return false;
    return true;
}

template <int FMT>
static cudaError_t launch_tree(const TreeMaps &tm, const TreeArgs &a, int grid, bool after, cudaStream_t st, int dev)
{
    static bool attr_done[64] = {};   // the attribute is set once per device
    if (dev >= 64 || !attr_done[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(tree_attn_kernel<FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(kTSmemBytes));
        if (e != cudaSuccess)
            return e;
        if (dev < 64)
            attr_done[dev] = true;
    }
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(FMT == EA_CACHE_BF16 ? kTThreads : kTThreadsQ8);
    cfg.dynamicSmemBytes = kTSmemBytes;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = after ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, tree_attn_kernel<FMT>, tm, a);
}

} // namespace ea

using namespace ea;

extern "C" size_t ea_tree_workspace_size(int B, int T, int Hq, int Hkv, int d, int Lmax)
{
    if (!tree_sizes_ok(B, T, Hq, Hkv, d) || Lmax < 1)
        return 0;
    return tree_ws_layout(B, T, Hq, Hkv, Lmax).total;
}

extern "C" ea_status ea_hybrid_attn_tree(const void *Q, const void *K, const void *V, const ea_cache *cache, void *O,
                                         float *LSE, const int64_t q_str[4], const int64_t kv_str[4],
                                         const int64_t o_str[4], const int32_t *seqlens, const int32_t *n_nodes,
                                         const int32_t *depth, const int32_t *mask, int B, int T, int Hq, float scale,
                                         const uint8_t *m, int sink, int window, const uint8_t *block_mask,
                                         int block_size, void *workspace, size_t ws_bytes, void *stream)
{
    if (!seqlens || !depth || !mask || !m || (reinterpret_cast<uintptr_t>(mask) & 15u))
        return EA_ERR_INVALID_ARG;
    TreeArgs a{};
    ea_status why;
    if (!cache_dev(cache, B, a.c, why))
        return why;
    const int Hkv = a.c.Hkv, Lmax = a.c.cap;
    if (T < 1 || Hq < 1 || Hq % Hkv != 0 || sink < 0 || window < 1 || !(scale > 0.f) || block_size != EA_TILE ||
        !tree_tensor(Q, q_str) || !tree_tensor(K, kv_str) || !tree_tensor(V, kv_str) || !tree_tensor(O, o_str))
        return EA_ERR_INVALID_ARG;
    const int64_t nBm = ceil_div(Lmax, EA_TILE);
    if (!tree_sizes_ok(B, T, Hq, Hkv, EA_HEAD_DIM) || (a.c.table && a.c.rows % 64) || (block_mask && nBm > 65535))
        return EA_ERR_UNSUPPORTED;
    const TreeWs w = tree_ws_layout(B, T, Hq, Hkv, Lmax);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || ws_bytes < w.total)
        return EA_ERR_WORKSPACE;

    a.g = Hq / Hkv;
    a.tpt = w.tpt;
    a.box128 = !a.c.table || a.c.rows % kTTile == 0;
    alignas(64) TreeMaps tm;
    const bool wide = a.c.format == EA_CACHE_BF16;
    if (!encode_tmap_bf16_rows(&tm.q, Q, Hq, T, B, q_str, a.g, a.tpt) ||
        !encode_tmap_bf16_rows(&tm.kd, K, Hkv, T, B, kv_str, 1, kTTile) ||
        !encode_tmap_bf16_rows(&tm.vd, V, Hkv, T, B, kv_str, 1, kTTile))
        return EA_ERR_INVALID_ARG;
    if (wide) {
        const int box = a.box128 ? kTTile : 64;
        if (!encode_tmap_bf16_rows(&tm.k, a.c.code[0], Hkv, a.c.rows, a.c.outer, cache->kv_str, 1, box) ||
            !encode_tmap_bf16_rows(&tm.v, a.c.code[1], Hkv, a.c.rows, a.c.outer, cache->kv_str, 1, box))
            return EA_ERR_INVALID_ARG;
    } else {
        tm.k = tm.kd;
        tm.v = tm.vd;
    }
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.O = static_cast<__nv_bfloat16 *>(O);
    a.o_sb = o_str[0];
    a.o_st = o_str[1];
    a.o_sh = o_str[2];
    a.LSE = LSE;
    a.seqlens = seqlens;
    a.n_nodes = n_nodes;
    a.depth = depth;
    a.mask = reinterpret_cast<const uint4 *>(mask);
    a.m = m;
    a.block_mask = block_mask;
    a.blk_count = reinterpret_cast<int32_t *>(ws + w.blk_count);
    a.blk_list = reinterpret_cast<uint32_t *>(ws + w.blk_list);
    a.first = reinterpret_cast<int32_t *>(ws + w.first);
    a.last = reinterpret_cast<int32_t *>(ws + w.last);
    a.part_lse = reinterpret_cast<float *>(ws + w.part_lse);
    a.part_o = reinterpret_cast<float *>(ws + w.part_o);
    a.hdr = reinterpret_cast<ea_ws_header *>(ws);
    a.B = B;
    a.T = T;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.pairs = w.pairs;
    a.rows_slot = w.rows_slot;
    a.nBm = static_cast<int>(nBm);
    // positions stay below 2^31 - 128: larger limits say the same
    a.sink = sink < (1 << 30) ? sink : 0x7fffffff;
    a.window = window;
    a.min_tiles = kTMinTiles;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.grow = kTGrow / a.scale_log2;

    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return EA_ERR_CUDA;
    const int sms = num_sms(dev);
    if (sms <= 0)
        return EA_ERR_CUDA;
    const int grid = sms < kTSms ? sms : kTSms;
    if (block_mask)
        tree_blocks_kernel<<<static_cast<unsigned>(B) * Hkv, kTBlkThreads, 0, st>>>(a);
    cudaError_t e;
    if (wide)
        e = launch_tree<EA_CACHE_BF16>(tm, a, grid, block_mask != nullptr, st, dev);
    else if (a.c.format == EA_CACHE_E4M3)
        e = launch_tree<EA_CACHE_E4M3>(tm, a, grid, block_mask != nullptr, st, dev);
    else
        e = launch_tree<EA_CACHE_INT8>(tm, a, grid, block_mask != nullptr, st, dev);
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg{};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = dim3(static_cast<unsigned>(ceil_div(static_cast<int64_t>(B) * T * Hq, kTMergeWarps)));
        cfg.blockDim = dim3(kTMergeWarps * 32);
        cfg.stream = st;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, tree_merge_kernel, a);
    }
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? EA_OK : EA_ERR_CUDA;
}
