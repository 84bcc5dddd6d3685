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
// HBM rate; an M tile takes 0.66 us of tensor core (at the measured bf16 rate) and 0.25 of the SFU.
// So HBM where one M tile does: 16 sequences of 64K with trees of 32 take 0.63 - 0.66 ms by GPU, 0.97 - 1.0 of
// the measured rate.  Two M tiles take 2.0 us a tile (0.87 - 0.89 ms with trees of 64, 1250 TFLOP/s), 1.3 of it tensor core:
// S = Q K^T, the softmax and O += P V of a tile wait for one another, and TMEM has no room for a
// second S of each.  An 8-bit cache's tile takes 1.3 us (0.59 ms with trees of 16, 0.54 of the
// measured rate): the same chain, beside the conversion.
//
// Work.  Key tiles of all (sequence, KV head, pair of M tiles) form one line, which is cut
// into equal ranges, one a CTA: no CTA idles, and at most two ranges of a CTA's begin or
// end inside a unit, so partial results are bounded by the grid, whatever the batch.  Every
// CTA finds its range itself (a scan over the units' tile counts).
//
// Roles of a CTA:
//   warps 0-7    two softmax warpgroups.  With two M tiles each has one; with one they take
//                key tiles in turn, each with its own O, m and l, joined at the range's end.
//   warp 8       the range, and by TMA the K and V tiles into a ring of 32 KB entries
//   warp 9       S = Q K^T
//   warp 10      O += P V
//   warp 11      Q, and V's rows that no query row keeps are zeroed before the product (0 * NaN is
//                NaN), and tiles of which some rows keep a key and others do not are searched
//                for infinities and NaN; such a tile's product is taken by the softmax warps,
//                key by key, as are 8-bit tiles whose scales are far apart (tree_convert)
//   warps 12-19  8-bit caches: tiles of codes, that TMA brought, become f16 ones in the ring
#include <cuda.h>
#include <cuda_runtime.h>

#include "ea_cache.cuh"
#include "ea_internal.h"

namespace ea {

constexpr int kTTile = 128;
constexpr int kTBytes = kTTile * EA_HEAD_DIM * 2;     // a tile of K, V or Q: 32 KB
constexpr int kTHalf = kTBytes / 2;                   // 64 dims of 128 rows
constexpr int kTInfos = 8;                            // tile descriptions in flight: the rings and S hold six tiles at most
constexpr int kTReady = 8;
constexpr int kTSegs = 3;
constexpr int kTProducerWarp = 8, kTQkWarp = 9, kTPvWarp = 10, kTConvWarp = 12, kTConvWarps = 8;
constexpr int kTThreads = kTConvWarp * 32, kTThreadsQ8 = (kTConvWarp + kTConvWarps) * 32;
constexpr uint32_t kTColO = 256;                      // TMEM: S0, S1, O0, O1
constexpr uint32_t kTIdescQK = idesc_bf16_f32(128, 128, false, false);
constexpr uint32_t kTIdescPV = idesc_bf16_f32(128, 128, false, true);
constexpr uint32_t kTIdescBf16 = 1u << 7 | 1u << 10;  // the operands' type: bf16; without these bits f16
constexpr float kTGrow = 8.f;                         // the maximum is followed once it grew by 2^8: p <= 2^8
constexpr float kTShift = 7.f;                        // 8-bit caches: p is f16, at most 2^(7 + 8)
constexpr int kTMinTiles = 2;                         // of a range at least (a power of two)
constexpr int kTPartTiles = 4;                        // see tree_range
constexpr int kTSpread = 12;                          // see tree_convert
constexpr int kTFewKeys = 512;                        // bf16 caches: P V in two parts up to these, see exp32_parts
constexpr int kTSms = 152;                            // a workspace's size depends on the grid

enum { kEdge = 1, kDraft = 2, kRow0 = 4, kRow1 = 8, kMixed = 16, kWide = 32, kGroups = 8 };   // (from bit 8 on: 16-key groups)

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
    int B, T, Hq, Hkv, g, tpt, pairs, nBm, sink, window, box128, rows_slot;
    int page_log2;                       // of a page size that is a power of two, else -1
    float inv_Hkv, inv_g, inv_tpt;       // for quot()
    float scale_log2;
};

struct TreeMaps {
    CUtensorMap q, kd, vd, k, v;
};

// x / d for 0 <= x < 2^24, inv = 1 / d (a division takes the start of a CTA ten times as long).
__device__ __forceinline__ int quot(int x, int d, float inv)
{
    const int q = __float2int_rz(static_cast<float>(x) * inv), r = x - q * d;
    return q + (r >= d ? 1 : 0) - (r < 0 ? 1 : 0);
}

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
    const int b = quot(u, a.Hkv, a.inv_Hkv);
    x.n = a.n_nodes ? __ldg(a.n_nodes + b) : a.T;
    x.L = __ldg(a.seqlens + b);
    x.mode = __ldg(a.m + u);
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
    x.pairs = x.n <= 0 ? 0 : a.pairs == 1 ? 1 : (quot(x.n + a.tpt - 1, a.tpt, a.inv_tpt) + 1) / 2;
    return x;
}

// A range's part of one unit.
struct TreeSeg {
    int valid;
    int b, h, v;                         // v: unit * pairs + pair
    int mode, L, n;
    bool dead, few;                      // no key is kept; no row keeps more than kTFewKeys of the cache
    int tok0, two;                       // first node, and whether there are two M tiles
    int t0, t1, nt;                      // tiles [t0, t1) of nt
    int slot;                            // of the partial result
};

struct TreeTile {
    int key0, flags;
    int outer[2], row[2];                // where its halves lie in the cache (row < 0: not read; outer < 0: zeros)
};

// The tile of the tree's own keys.
__device__ __forceinline__ TreeTile tree_own_tile(int L, int n)
{
    return TreeTile{L, kEdge | kDraft | kMixed | ((n + 15) / 16) << kGroups, {0, 0}, {0, 0}};
}

__device__ __forceinline__ TreeTile tree_tile(const TreeArgs &a, const TreeUnit &x, int u, int t)
{
    TreeTile r{};
    if (t >= x.nt - 1)
        return tree_own_tile(x.L, x.n);
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
    r.flags |= ((min(kTTile, x.L - r.key0) + 15) / 16) << kGroups;
    return r;
}

// Shared memory is what bounds the bytes on their way: a second M tile's queries take one
// ring entry's place, and an 8-bit cache's codes two.
template <bool Q8_, bool TWO>
struct __align__(1024) TreeSmem {
    static constexpr bool Q8 = Q8_;
    static constexpr int kStages = Q8 ? 4 : TWO ? 5 : 6;       // ring entries: K or V tiles, in turn
    static constexpr int kCodes = Q8 ? (TWO ? 2 : 4) : 1;      // tiles of codes, K and V in turn
    uint8_t q[TWO ? 2 : 1][kTBytes];
    uint8_t ring[kStages][kTBytes];
    uint8_t code[kCodes][Q8 ? kTBytes / 2 : 16];
    float2 ml[Q8 ? 1 : 2][kTTile];       // a warpgroup's maximum and sum of each row; before: the scan
    uint64_t full[kStages], empty[kStages];
    uint64_t code_full[kCodes], code_empty[kCodes];
    uint64_t ready[kTReady];             // V has been looked over
    uint64_t seg_full[kTSegs], seg_empty[kTSegs];
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_full[2], o_done[2];
    uint64_t seg_done, ml_full[2], o_free, drain;
    uint64_t q_ready, own_full[2], own_max[2];   // 8-bit caches: Q in f16; the tree's K and V
    TreeSeg seg[kTSegs];
    TreeTile tile[kTInfos];
    // 8-bit caches: a 16-key group's (K's, V's) and a drafted key's f16 numbers stand for 2^(unit - 127) times them (a
    // group of the tree's own rows: 0 if those have units of their own)
    alignas(16) uint8_t group_unit[Q8 ? kTInfos : 1][2][8];
    uint8_t own_unit[Q8 ? kTSegs : 1][2][Q8 ? kTTile : 1];
    uint8_t own_exp[2][2][2][4];         // the largest and the least exponent of a warp's drafted rows
    uint8_t odd[kTReady];                // V holds an infinity or a NaN
    TreeUnit unit;                       // this CTA's range: its first unit,
    int u, off, count;                   // where it starts in it, and its tiles
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(TreeSmem<false, false>) <= 232448 && sizeof(TreeSmem<false, true>) <= 232448 &&
                  sizeof(TreeSmem<true, false>) <= 232448 && sizeof(TreeSmem<true, true>) <= 232448,
              "shared memory of one CTA");

// The tensor core's instructions where `go` is set (one thread of the warp): predicated, not
// branched around, so that the warp's flow stays uniform.
__device__ __forceinline__ void mma_ss(uint32_t go, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(go)
                 : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t go, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(go)
                 : "memory");
}

__device__ __forceinline__ void commit_if(uint32_t go, uint64_t *bar)
{
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
                 "r"(go)
                 : "memory");
}

__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}

// 32 lanes x 16 columns of 32-bit TMEM -> 16 registers per thread.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr)
                 : "memory");
}

// Keeps the registers of a TMEM load behind the wait for it (the compiler sees no
// dependence between the two).
__device__ __forceinline__ void tie32(uint32_t (&r)[32])
{
#pragma unroll
    for (int i = 0; i < 32; ++i)
        asm volatile("" : "+r"(r[i]));
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

// Part number `it` of the range (in slot it % kTSegs, held until tree_done), by a whole warp; NULL: none
// left, or gave up.
template <class Smem>
__device__ __forceinline__ const TreeSeg *tree_take(const TreeArgs &a, Smem &sm, uint32_t it)
{
    const int slot = it % kTSegs;
    if (!mbar_wait_warp(&sm.seg_full[slot], (it / kTSegs) & 1, &sm.abort, &a.hdr->error))
        return nullptr;
    return sm.seg[slot].valid ? &sm.seg[slot] : nullptr;
}

template <class Smem>
__device__ __forceinline__ void tree_done(Smem &sm, uint32_t it)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(&sm.seg_empty[it % kTSegs]);
}

// ------------------------------------------------------------ ranges
// This CTA's range: an equal share of the line of tiles among G CTAs (fewer than the grid where a share
// would be shorter than kTMinTiles).  A unit's queries, its own keys and its results cost about as much
// as kTPartTiles of its tiles, which lie ahead of them in the line (eight int8 sequences, of 30000 keys
// and of none: 101 -> 55 us).  Found by one warp where there are few units, so that the others'
// set-up runs beside it; by all of them (ahead of their roles) else.
constexpr int kTWarpUnits = 256;

template <class Smem>
__device__ __forceinline__ void tree_range(const TreeArgs &a, Smem &sm, int tid, int warps)
{
    const int lane = tid & 31, warp = tid / 32, units = a.B * a.Hkv;
    const int per = units <= 32 ? 1 : (units + 32 * warps - 1) / (32 * warps);
    const int lo = min(tid * per, units), hi = min(lo + per, units);
    int mine = 0;
    bool bad = false;
    TreeUnit x{};
    for (int u = lo; u < hi; ++u) {
        x = tree_unit(a, u);
        mine += (x.nt + kTPartTiles) * x.pairs;
        bad |= x.bad;
    }
    if (bad && blockIdx.x == 0)
        raise_error(&a.hdr->error, EA_DEVERR_CHECK);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += v;
    }
    int before = 0, W = __shfl_sync(0xffffffffu, incl, 31);
    if (tid == 0)
        sm.count = 0;
    if (warps > 1) {
        int *tot = reinterpret_cast<int *>(sm.ml);
        if (lane == 31)
            tot[warp] = incl;
        __syncthreads();
        W = 0;
        for (int w = 0; w < warps; ++w) {
            before += w < warp ? tot[w] : 0;
            W += tot[w];
        }
    } else {
        __syncwarp();
    }
    int base = before + incl - mine;
    const int G = max(1, min(static_cast<int>(gridDim.x), W / kTMinTiles));
    const int i = blockIdx.x, share = W / G, rest = W - share * G;
    const int start = i * share + min(i, rest), count = share + (i < rest ? 1 : 0);
    if (i < G && count > 0 && start >= base && start < base + mine)
        for (int u = lo; u < hi; ++u) {
            if (per > 1)
                x = tree_unit(a, u);
            const int w = (x.nt + kTPartTiles) * x.pairs;
            if (start < base + w) {
                sm.unit = x;
                sm.u = u;
                sm.off = start - base;
                sm.count = count;
                break;
            }
            base += w;
        }
}

// ------------------------------------------------------------ K and V
// Where 64 keys of a tile lie in the cache; row < 0: behind the sequence (not read).
__device__ __forceinline__ void tree_place(const TreeArgs &a, int b, int L, int key, int &outer, int &row)
{
    outer = b;
    row = key < L ? key : -1;
    if (row >= 0 && a.c.table) {
        const int pg = a.page_log2 >= 0 ? key >> a.page_log2 : key / a.c.rows;
        row = key - pg * a.c.rows;
        outer = a.c.table[b * a.c.bt_stride + pg];
        if (outer < 0 || outer >= a.c.outer) {         // reported; reads zeros
            raise_error(&a.hdr->error, EA_DEVERR_CHECK);
            outer = -1;
        }
    }
}

// K or V of the tree's own tokens (rows behind the tensor read zeros).
__device__ __forceinline__ void tree_load_own(const TreeMaps &tm, uint8_t *dst, int kv, const TreeSeg &s, uint64_t *bar)
{
    mbar_arrive_expect_tx(bar, kTBytes);
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
        tma_load_4d(dst + hf * kTHalf, kv ? &tm.vd : &tm.kd, 64 * hf, s.h, 0, s.b, bar);
}

template <class Smem>
__device__ __forceinline__ void tree_producer(const TreeMaps &tm, const TreeArgs &a, Smem &sm, int lane)
{
    constexpr bool Q8 = Smem::Q8;
    constexpr int kStages = Smem::kStages, kCodes = Smem::kCodes;
    uint32_t *err = &a.hdr->error;
    int u = sm.u, off = sm.off, left = sm.count;
    TreeUnit x = sm.unit;                // the unit at hand
    uint32_t it = 0, entry = 0, codes = 0, tile = 0;
    bool ok = true;
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
        const int len = x.nt + kTPartTiles;
        if (off >= len * x.pairs) {
            x = tree_unit(a, ++u);
            off = 0;
            continue;
        }
        TreeSeg s;
        // the rest of one pair of M tiles, as far as the range goes
        const int pair = x.pairs == 1 ? 0 : off / len, from = off - pair * len, to = left < len - from ? from + left : len;
        off += to - from;
        left -= to - from;
        if (to <= kTPartTiles)
            continue;
        s.valid = 1;
        s.b = quot(u, a.Hkv, a.inv_Hkv);
        s.h = u - s.b * a.Hkv;
        s.v = u * a.pairs + pair;
        s.mode = x.mode;
        s.L = x.L;
        s.n = x.n;
        s.dead = x.dead;
        if constexpr (!Q8) {
            // (the window of depth 0; of a block row's last block one key at least)
            const int kept = x.mode == EA_FULL ? x.L : x.mode == EA_SSA ? x.n0 + x.L - max(x.n0, x.L - a.window + 1) : (x.nt - 2) * kTTile + 1;
            s.few = kept <= kTFewKeys;
        }
        s.tok0 = 2 * pair * a.tpt;
        s.two = s.tok0 + a.tpt < x.n;
        s.t0 = max(from - kTPartTiles, 0);
        s.t1 = to - kTPartTiles;
        s.nt = x.nt;
        // a range holds one part that continues a unit (its first) and one that is continued at most
        s.slot = 2 * blockIdx.x + (s.t0 == 0 ? 1 : 0);
        if (!publish(s))
            break;
        if (lane == 0) {
            if (s.t0 == 0)
                a.first[s.v] = blockIdx.x;
            if (s.t1 == s.nt)
                a.last[s.v] = blockIdx.x;
        }
        __syncwarp();
        ++it;
        // Lanes 2 i and 2 i + 1 hold the places of the halves of tile i of sixteen.
        TreeTile mine{};
        int row = -1, outer = 0;
        for (int t = s.t0; t < s.t1; ++t, ++tile) {
            const int i = (t - s.t0) & 15;
            if (i == 0) {
                const int tt = t + (lane >> 1);
                uint32_t hi[2] = {0u, 0u}, lo[2] = {255u, 255u};
                if (tt < s.t1) {
                    mine = tree_tile(a, x, u, tt);
                    if (!(mine.flags & kDraft)) {
                        tree_place(a, s.b, s.L, mine.key0 + 64 * (lane & 1), outer, row);
                        if (Q8 && row >= 0 && outer >= 0) {
                            // how far their scales are apart (and in L1 for the converting warps)
                            const int64_t at = (static_cast<int64_t>(outer) * a.c.Hkv + s.h) * a.c.nsb;
                            uint32_t w[2][4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int p = min(row + 16 * i, row + s.L - 1 - (mine.key0 + 64 * (lane & 1))) >> a.c.log2sb;
#pragma unroll
                                for (int kv = 0; kv < 2; ++kv)
                                    w[kv][i] = __ldg(reinterpret_cast<const uint32_t *>(a.c.scale[kv]) + at + p);
                            }
#pragma unroll
                            for (int kv = 0; kv < 2; ++kv)
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const uint32_t e = (w[kv][i] & 0x7fffffffu) >= 0x7f800000u ? 0u : w[kv][i] >> 23;
                                    hi[kv] = max(hi[kv], e);
                                    lo[kv] = e > 127u - 64u ? min(lo[kv], e) : lo[kv];
                                }
                        }
                    }
                }
                __syncwarp();
                if constexpr (Q8) {
                    // (of both halves)
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const uint32_t top = max(hi[kv], __shfl_xor_sync(0xffffffffu, hi[kv], 1)), low = min(lo[kv], __shfl_xor_sync(0xffffffffu, lo[kv], 1));
                        if (top > low + kTSpread)
                            mine.flags |= kWide;
                    }
                }
            }
            TreeTile ti;
            ti.key0 = __shfl_sync(0xffffffffu, mine.key0, 2 * i);
            ti.flags = __shfl_sync(0xffffffffu, mine.flags, 2 * i);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                ti.row[hf] = __shfl_sync(0xffffffffu, row, 2 * i + hf);
                ti.outer[hf] = __shfl_sync(0xffffffffu, outer, 2 * i + hf);
            }
            if constexpr (Q8) {
                // the codes; the converting warps fill the ring (with the tree's own keys too)
#pragma unroll
                for (int kv = 0; kv < 2 && !(ti.flags & kDraft); ++kv, ++codes) {
                    const int cs = codes % kCodes;
                    if (!mbar_wait_warp(&sm.code_empty[cs], ((codes / kCodes) & 1) ^ 1, &sm.abort, err)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        if (kv == 0)
                            sm.tile[tile % kTInfos] = ti;
                        uint64_t *bar = &sm.code_full[cs];
                        const CUtensorMap *map = kv ? &tm.v : &tm.k;
                        mbar_arrive_expect_tx(bar, (a.box128 || ti.row[1] >= 0) ? kTBytes / 2 : kTBytes / 4);
                        tma_load_4d(sm.code[cs], map, 0, s.h, ti.row[0], ti.outer[0], bar);
                        if (!a.box128 && ti.row[1] >= 0)
                            tma_load_4d(sm.code[cs] + kTBytes / 4, map, 0, s.h, ti.row[1], ti.outer[1], bar);
                    }
                    __syncwarp();
                }
            } else {
#pragma unroll
            for (int kv = 0; kv < 2; ++kv, ++entry) {
                const int st = entry % kStages;
                if (!mbar_wait_warp(&sm.empty[st], ((entry / kStages) & 1) ^ 1, &sm.abort, err)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    uint8_t *dst = sm.ring[st];
                    uint64_t *bar = &sm.full[st];
                    if (kv == 0)
                        sm.tile[tile % kTInfos] = ti;
                    if (ti.flags & kDraft) {
                        tree_load_own(tm, dst, kv, s, bar);
                    } else if (a.box128) {
                        mbar_arrive_expect_tx(bar, kTBytes);
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf)
                            tma_load_4d(dst + hf * kTHalf, kv ? &tm.v : &tm.k, 64 * hf, s.h, ti.row[0], ti.outer[0], bar);
                    } else {
                        mbar_arrive_expect_tx(bar, ti.row[1] >= 0 ? kTBytes : kTHalf);
#pragma unroll
                        for (int p = 0; p < 2; ++p)
                            if (ti.row[p] >= 0)
#pragma unroll
                                for (int hf = 0; hf < 2; ++hf)
                                    tma_load_4d(dst + hf * kTHalf + p * (kTHalf / 2), kv ? &tm.v : &tm.k, 64 * hf, s.h,
                                                ti.row[p], ti.outer[p], bar);
                    }
                }
                __syncwarp();
            }
            }
            if (!ok)
                break;
        }
    }
    TreeSeg none{};
    if (ok)
        publish(none);
    // Before leaving on an abort, let the copies already issued land.
    if (__any_sync(0xffffffffu, *static_cast<volatile int *>(&sm.abort))) {
        volatile int no_abort = 0;
        if constexpr (Q8)
            for (uint32_t n = codes > kCodes ? codes - kCodes : 0; n < codes; ++n)
                mbar_wait_warp(&sm.code_full[n % kCodes], (n / kCodes) & 1, &no_abort, nullptr);
        for (uint32_t n = entry > kStages ? entry - kStages : 0; n < entry; ++n)
            mbar_wait_warp(&sm.full[n % kStages], (n / kStages) & 1, &no_abort, nullptr);
    }
}

// ------------------------------------------------------------ products
// Two warps, one for S = Q K^T and one for O += P V (an issue with its waits and commits takes one warp
// about 1000 cycles, as long as the products take: one warp for both paced the kernel), one thread of
// each for the MMAs.  The warps stay whole and their values uniform, so that the operands' descriptors
// are worked out in uniform registers: in one thread's own branch, eight MMAs took 750 cycles to issue.
template <class Smem>
__device__ __forceinline__ void tree_qk(const TreeArgs &a, Smem &sm, uint32_t tmem_base)
{
    constexpr int kStages = Smem::kStages;
    constexpr bool TWO = sizeof(sm.q) > kTBytes;
    constexpr uint32_t kIdQK = (Smem::Q8 ? kTIdescQK & ~kTIdescBf16 : kTIdescQK) & ~(63u << 17);
    volatile int *abort = &sm.abort;
    uint32_t *err = &a.hdr->error;
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
    const uint64_t q0 = sdesc_sw128(smem_u32(sm.q[0]), 16, 1024), ring0 = sdesc_sw128(smem_u32(sm.ring[0]), 16, 1024);
    const uint32_t go = elect_one();
    uint32_t tile0 = 0, cnt[2] = {0, 0};
    const TreeSeg *sp;
    for (uint32_t it = 0; (sp = tree_take(a, sm, it)) != nullptr; ++it) {
        const int two = TWO ? __shfl_sync(0xffffffffu, sp->two, 0) : 0;
        const int nt = __shfl_sync(0xffffffffu, sp->t1 - sp->t0, 0);
        if (!mbar_wait_warp(Smem::Q8 ? &sm.q_ready : &sm.q_full, it & 1, abort, err))
            break;
        const int N = nt << two;
        for (int n = 0; n < N; ++n) {
            const int w = n & 1;
            const uint32_t tile = tile0 + (n >> two), e = 2 * tile;
            const int st = e % kStages;
            const uint64_t qd = q0 + static_cast<uint64_t>((two & w) * (kTBytes >> 4));
            const uint64_t kd = ring0 + static_cast<uint64_t>(st * (kTBytes >> 4));
            const uint32_t ts = tmem + 128 * w;
            // K, and this S's last user, the product two steps before
            bool in = mbar_wait(&sm.full[st], (e / kStages) & 1, abort, err);
            in = in && (cnt[w] == 0 || mbar_wait(&sm.o_done[w], (cnt[w] - 1) & 1, abort, err));
            if (!__all_sync(0xffffffffu, in))
                break;
            ++cnt[w];
            tc_fence_after();
            // (a tile with fewer keys: the columns behind them are masked)
            const uint32_t id = kIdQK | static_cast<uint32_t>(__shfl_sync(0xffffffffu, sm.tile[tile % kTInfos].flags >> kGroups, 0)) << 18;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint64_t o = ((k >> 2) * kTHalf + (k & 3) * 32) >> 4;
                mma_ss(go, ts, qd + o, kd + o, id, k > 0);
            }
            commit_if(go, &sm.s_full[w]);
            if (!two || w == 1)
                commit_if(go, &sm.empty[st]);
            if (n == N - 1)
                commit_if(go, &sm.q_empty);
        }
        tile0 += nt;
        tree_done(sm, it);
    }
    // All of this warp's MMAs must have completed before TMEM is released.
    commit_if(go, &sm.drain);
    volatile int no_abort = 0;
    mbar_wait_warp(&sm.drain, 0, &no_abort, err);
}

template <class Smem>
__device__ __forceinline__ void tree_pv(const TreeArgs &a, Smem &sm, uint32_t tmem_base)
{
    constexpr int kStages = Smem::kStages;
    constexpr bool TWO = sizeof(sm.q) > kTBytes;
    constexpr uint32_t kIdPV = Smem::Q8 ? kTIdescPV & ~kTIdescBf16 : kTIdescPV;
    volatile int *abort = &sm.abort;
    uint32_t *err = &a.hdr->error;
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
    const uint64_t ring0 = sdesc_sw128(smem_u32(sm.ring[0]), kTHalf, 1024);
    const uint32_t go = elect_one();
    uint32_t tile0 = 0, cnt[2] = {0, 0};
    const TreeSeg *sp;
    for (uint32_t it = 0; (sp = tree_take(a, sm, it)) != nullptr; ++it) {
        const int two = TWO ? __shfl_sync(0xffffffffu, sp->two, 0) : 0;
        const int nt = __shfl_sync(0xffffffffu, sp->t1 - sp->t0, 0);
        const int few = Smem::Q8 ? 0 : __shfl_sync(0xffffffffu, sp->few, 0);
        // (O is still read for the range's part before)
        if (it > 0 && !mbar_wait_warp(&sm.o_free, (it - 1) & 1, abort, err))
            break;
        const int N = nt << two;
        for (int n = 0; n < N; ++n) {
            const int w = n & 1;
            const uint32_t tile = tile0 + (n >> two), e = 2 * tile + 1;
            const int st = e % kStages;
            const uint64_t vd = ring0 + static_cast<uint64_t>(st * (kTBytes >> 4));
            const uint32_t tp = tmem + 128 * w, to = tmem + kTColO + 128 * w;
            // (a warpgroup's first product of the range overwrites what its O held)
            const uint32_t more = n >= 2;
            bool in = mbar_wait(&sm.ready[tile % kTReady], (tile / kTReady) & 1, abort, err);
            const int flags = __shfl_sync(0xffffffffu, sm.tile[tile % kTInfos].flags, 0);
            const int odd = __shfl_sync(0xffffffffu, static_cast<int>(sm.odd[tile % kTReady]), 0);
            in = in && mbar_wait(&sm.p_full[w], cnt[w] & 1, abort, err);
            if (!__all_sync(0xffffffffu, in))
                break;
            ++cnt[w];
            tc_fence_after();
            if (!(flags & kEdge) && !odd) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mma_ts(go, to, tp + 32 * (k >> 1) + 8 * (k & 1), vd + k * (2048 >> 4), kIdPV, k ? 1u : more);
            } else if (!odd) {
                const int groups = flags >> kGroups;
#pragma unroll 1
                for (int k = 0; k < groups; ++k)
                    mma_ts(go, to, tp + 32 * (k >> 1) + 8 * (k & 1), vd + k * (2048 >> 4), kIdPV, k ? 1u : more);
            }
            if (few && !odd) {
                // P's second part
                const int groups = flags >> kGroups;
#pragma unroll 2
                for (int k = 0; k < groups; ++k)
                    mma_ts(go, to, tp + 32 * (k >> 1) + 8 * (k & 1) + 16, vd + k * (2048 >> 4), kIdPV, 1u);
            }
            commit_if(go, &sm.o_done[w]);
            if (!two || w == 1)
                commit_if(go, &sm.empty[st]);
            if (n == N - 1)
                commit_if(go, &sm.seg_done);
        }
        tile0 += nt;
        tree_done(sm, it);
    }
    commit_if(go, &sm.drain);
    volatile int no_abort = 0;
    mbar_wait_warp(&sm.drain, 0, &no_abort, err);
}

// ------------------------------------------------------------ V's rows
// An infinity or a NaN among two bf16 (f16) numbers.
template <bool F16>
__device__ __forceinline__ bool odd2(uint32_t w)
{
    constexpr uint32_t kLo = F16 ? 0x7c00u : 0x7f80u, kHi = kLo << 16;
    return (w & kLo) == kLo || (w & kHi) == kHi;
}

template <class Smem>
__device__ __forceinline__ void tree_fix(const TreeMaps &tm, const TreeArgs &a, Smem &sm, int lane)
{
    constexpr int kStages = Smem::kStages;
    uint32_t *err = &a.hdr->error;
    uint32_t tile = 0, it = 0;
    for (const TreeSeg *sp; (sp = tree_take(a, sm, it)) != nullptr; ++it) {
        const TreeSeg &s = *sp;
        // the queries
        if (!mbar_wait_warp(&sm.q_empty, (it & 1) ^ 1, &sm.abort, err))
            break;
        if (lane == 0) {
            const int tiles = sizeof(sm.q) > kTBytes && s.two ? 2 : 1;
            mbar_arrive_expect_tx(&sm.q_full, static_cast<uint32_t>(tiles * a.g * a.tpt) * 256u);
            for (int w = 0; w < tiles; ++w)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
                    tma_load_4d(sm.q[w] + hf * kTHalf, &tm.q, 64 * hf, s.h * a.g, s.tok0 + w * a.tpt, s.b, &sm.q_full);
        }
        __syncwarp();
        for (int t = s.t0; t < s.t1; ++t, ++tile) {
            const uint32_t e = 2 * tile;
            const int ks = e % kStages, vs = (e + 1) % kStages;
            if (!mbar_wait_warp(&sm.full[ks], (e / kStages) & 1, &sm.abort, err))
                break;
            const TreeTile ti = sm.tile[tile % kTInfos];
            if (!mbar_wait_warp(&sm.full[vs], ((e + 1) / kStages) & 1, &sm.abort, err))
                break;
            bool odd = false;
            if (ti.flags & kEdge) {
                const int nv = (ti.flags & kDraft) ? s.n : min(kTTile, s.L - ti.key0);
                const int from = (ti.flags & kMixed) ? 0 : nv * 16;
                // 16 bytes of row i / 16: eight of each half (their order in a row does not matter)
#pragma unroll 4
                for (int i = from + lane; i < (ti.flags >> kGroups) * 256; i += 32) {
                    uint4 *p = reinterpret_cast<uint4 *>(sm.ring[vs] + ((i >> 3) & 1) * kTHalf + (i >> 4) * 128 + (i & 7) * 16);
                    if ((i >> 4) >= nv) {
                        *p = make_uint4(0u, 0u, 0u, 0u);
                    } else {
                        const uint4 v = *p;
                        odd |= odd2<Smem::Q8>(v.x) | odd2<Smem::Q8>(v.y) | odd2<Smem::Q8>(v.z) | odd2<Smem::Q8>(v.w);
                    }
                }
                fence_proxy_async_smem();
            }
            // (rows with units of their own are taken key by key too)
            if (Smem::Q8)
                odd |= (ti.flags & kWide) || sm.group_unit[tile % kTInfos][0][0] == 0 || sm.group_unit[tile % kTInfos][1][0] == 0;
            odd = __any_sync(0xffffffffu, odd);
            if (lane == 0) {
                sm.odd[tile % kTReady] = odd;
                mbar_arrive(&sm.ready[tile % kTReady]);
                mbar_arrive(&sm.empty[ks]);
                mbar_arrive(&sm.empty[vs]);
            }
            __syncwarp();
        }
        tree_done(sm, it);
    }
    // Before leaving on an abort, let the queries already issued land.
    if (it > 0 && __any_sync(0xffffffffu, *static_cast<volatile int *>(&sm.abort))) {
        volatile int no_abort = 0;
        mbar_wait_warp(&sm.q_full, (it - 1) & 1, &no_abort, nullptr);
    }
}

// ------------------------------------------------------------ 8-bit caches
// A tile of codes becomes f16.  Where its scales lie within 2^kTSpread of one another, a code times 2^(e - E + kTHead), e
// its block's exponent and E the largest of the tile's, so that one factor, 2^(E - kTHead), says what the tile's numbers
// stand for.  They are exact, and the softmax's weights, scaled to f16's upper end with the largest scale, lose kTSpread bits
// of its lower end at most, whatever lies in the tile that a row does not keep.  Else a code times 2^kTHead, a unit each 16
// keys, and the softmax takes the tile key by key.  (Units of 16 keys in every tile's softmax: 16 sequences of 64K, trees of 16,
// e4m3 574 -> 630 us; a path of its own for such tiles beside it, which no other tile runs, 592.)  The smallest scale,
// 2^-64, which a block of zeros has, counts for nothing: beside one above 2^-52 its numbers may become zero (as a drafted
// row below 2^-63).
// The tree's own rows, bf16, take one power of two, or, where their largest elements are further than 2^kTSpread apart, each
// its own, and go key by key too.
//   e4m3: two codes a conversion, then a multiplication
//   int8: c + 128 in the fraction of 1024, then (1024 + c + 128) f - 1152 f
template <bool E4M3>
constexpr int kTHead = E4M3 ? 6 : 5;

template <bool E4M3>
__device__ __forceinline__ uint2 codes_scaled(uint32_t w, __half2 f, __half2 g)
{
    __half2 x, y;
    if constexpr (E4M3) {
        uint32_t lo, hi;
        codes_f16<true>(w, lo, hi);
        x = __hmul2(*reinterpret_cast<const __half2 *>(&lo), f);
        y = __hmul2(*reinterpret_cast<const __half2 *>(&hi), f);
    } else {
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
        x = __hfma2(*reinterpret_cast<const __half2 *>(&lo), f, g);
        y = __hfma2(*reinterpret_cast<const __half2 *>(&hi), f, g);
    }
    return make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
}

__device__ __forceinline__ float pow2f(int e)          // -126 .. 127
{
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// The largest magnitude among eight bf16 numbers and `m`; NaN do not count.
__device__ __forceinline__ float max_mag(const uint4 &v, float m)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = max3f(m, __uint_as_float((w[i] << 16) & 0x7fffffffu), __uint_as_float(w[i] & 0x7fff0000u));
    return m;
}

// The same without infinities.
__device__ __forceinline__ float max_finite(const uint4 &v, float m)
{
    const uint32_t w[8] = {v.x << 16, v.x, v.y << 16, v.y, v.z << 16, v.z, v.w << 16, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = __uint_as_float(w[i] & 0x7fff0000u);
        m = x < __uint_as_float(0x7f800000u) ? fmaxf(m, x) : m;
    }
    return m;
}

// The biased exponent of a non-negative number.
__device__ __forceinline__ int exponent_of(float x)
{
    return static_cast<int>(__float_as_uint(x) >> 23);
}

// Eight bf16 numbers times f as f16.
__device__ __forceinline__ uint4 bf16_to_f16(const uint4 &v, float f)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xffff0000u) * f);
        o[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Warps that turn tiles of codes into the ring's f16 ones, four for K and four for V, so that the
// latencies of one (its codes, its scales, the fence) lie under the other's work.  A thread has 8
// codes of either half of eight rows, one row of each 16-key group, so lane i holds the scale of group
// i.  They become 16 bytes of the row in either half of the tile, swizzled as TMA would (odd rows'
// lanes take the second half first: two rows' codes then lie in different banks).
// A row an iteration, the next one's codes under its work: five roles take turns on a scheduler, and
// what bounded them when their loops were unrolled was instruction fetch (16 sequences of 64K: 680 us
// with the rows unrolled here and half of the columns in the softmax, 587 now).
template <bool E4M3, class Smem>
__device__ __forceinline__ void tree_convert(const TreeMaps &tm, const TreeArgs &a, Smem &sm, int kv, int ct, int lane)
{
    constexpr int kStages = Smem::kStages, kCodes = Smem::kCodes;
    static_assert(kStages % 2 == 0 && kCodes % 2 == 0, "a stage belongs to K or to V");
    uint32_t *err = &a.hdr->error;
    uint32_t entry = kv, codes = kv, tile = 0, own = 1;          // (own: one more than loads issued)
    const int piece = ct & 7, r0 = ct >> 3, flip = r0 & 1;
    const uint32_t in0 = r0 * 128 + 64 * flip + 8 * piece, in1 = in0 ^ 64u;
    const uint32_t at0 = flip * kTHalf + r0 * 128 + ((piece ^ (r0 & 7)) << 4), at1 = at0 ^ static_cast<uint32_t>(kTHalf);
    // lanes 0 - 7 look up this warp's scales; K's warps look up V's too (8 - 15), for the tile's factors
    const float *scales = a.c.scale[kv ^ (lane >> 3 & 1)];
    bool ok = true;
    for (uint32_t it = 0; ok; ++it) {
        const TreeSeg *sp = tree_take(a, sm, it);
        if (!sp)
            break;
        const TreeSeg &s = *sp;
        for (int t = s.t0; t < s.t1; ++t, ++tile, entry += 2) {
            const int st = entry % kStages, cs = codes % kCodes;
            uint8_t *dst = sm.ring[st];
            if (t == s.nt - 1) {
                // the tree's own: from bf16, a thread a row, times the power of two that puts its largest below 2^15
                if (!mbar_wait_warp(&sm.empty[st], ((entry / kStages) & 1) ^ 1, &sm.abort, err)) {
                    ok = false;
                    break;
                }
                if (ct == 0)
                    tree_load_own(tm, dst, kv, s, &sm.own_full[kv]);
                ++own;
                __syncwarp();
                if (!mbar_wait_warp(&sm.own_full[kv], own & 1, &sm.abort, err)) {
                    ok = false;
                    break;
                }
                auto part = [&](int c) { return reinterpret_cast<uint4 *>(dst + (c >> 3) * kTHalf + ct * 128 + (((c & 7) ^ (ct & 7)) << 4)); };
                float mx = 0.f;
                if (ct < s.n)
#pragma unroll 8
                    for (int c = 0; c < 16; ++c)
                        mx = max_finite(*part(c), mx);
                // (a row's largest counts as 2^-64 at least, a cache's smallest scale: sums of weights over V's unit stay
                // finite where V is zero)
                const int ex = max(exponent_of(mx), 127 - 64);
                const int hi = __reduce_max_sync(0xffffffffu, ct < s.n ? ex : 0), lo = __reduce_min_sync(0xffffffffu, ct < s.n && ex > 127 - 64 ? ex : 255);
                if (lane == 0) {
                    sm.own_exp[own & 1][kv][0][ct / 32] = static_cast<uint8_t>(hi);
                    sm.own_exp[own & 1][kv][1][ct / 32] = static_cast<uint8_t>(lo);
                    mbar_arrive(&sm.own_max[kv]);
                }
                __syncwarp();
                if (!mbar_wait_warp(&sm.own_max[kv], own & 1, &sm.abort, err)) {
                    ok = false;
                    break;
                }
                int top = 0, low = 255;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    top = max(top, static_cast<int>(sm.own_exp[own & 1][kv][0][i]));
                    low = min(low, static_cast<int>(sm.own_exp[own & 1][kv][1][i]));
                }
                const bool wide = top - low > kTSpread;
                const int unit = (wide ? ex : top) - 14;
                // (the slot's last user was the part three before, that all are through with)
                sm.own_unit[it % kTSegs][kv][ct] = static_cast<uint8_t>(unit);
                if (ct < 8)
                    sm.group_unit[tile % kTInfos][kv][ct] = static_cast<uint8_t>(wide ? 0 : unit);
                const float f = pow2f(127 - unit);
                asm volatile("" ::: "memory");           // (read again, not kept)
                if (ct < ((s.n + 15) & ~15))
#pragma unroll 8
                    for (int c = 0; c < 16; ++c)
                        *part(c) = bf16_to_f16(*part(c), f);
                if (ct == 0 && kv == 0)
                    sm.tile[tile % kTInfos] = tree_own_tile(s.L, s.n);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sm.full[st]);
                continue;
            }
            if (!mbar_wait_warp(&sm.code_full[cs], (codes / kCodes) & 1, &sm.abort, err)) {
                ok = false;
                break;
            }
            const TreeTile &ti = sm.tile[tile % kTInfos];
            uint32_t f = 0u;                           // a group's scale; none behind the end or outside the cache
            {
                const int i = lane & 7, hf = i >> 2, outer = ti.outer[hf], row = ti.row[hf] + 16 * (i & 3);
                if (lane < (kv ? 8 : 16) && outer >= 0 && ti.key0 + 16 * i < s.L)
                    f = __ldg(reinterpret_cast<const uint32_t *>(scales) +
                              (static_cast<int64_t>(outer) * a.c.Hkv + s.h) * a.c.nsb + (row >> a.c.log2sb));
            }
            const int groups = ti.flags >> kGroups;
            codes += 2;
            // the exponents (lanes 0 - 7, and V's in K's warps) and the largest
            const bool nan = (f & 0x7fffffffu) >= 0x7f800000u;
            const int e = nan ? 0 : static_cast<int>(f >> 23);
            int E = __reduce_max_sync(0xffffffffu, lane < 8 ? e : 0);
            const bool wide = (ti.flags & kWide) != 0;
            const int x = max(wide ? 0 : e - E, -100) + kTHead<E4M3>;
            if (kv == 0) {
                const int EV = __reduce_max_sync(0xffffffffu, lane >= 8 ? e : 0);
                E = lane < 8 ? E : EV;
                if (ct < 16)
                    sm.group_unit[tile % kTInfos][ct >> 3][ct & 7] =
                        static_cast<uint8_t>(max(wide ? e : E, 127 - 64) - kTHead<E4M3>);
            }
            // (a page outside the cache reads zeros, a block of a NaN scale NaN)
            uint32_t fg;
            {
                const __half h = nan ? __ushort_as_half(0x7e00) : __float2half_rn(e ? pow2f(x) : 0.f);
                fg = static_cast<uint32_t>(__half_as_ushort(h)) |
                     static_cast<uint32_t>(__half_as_ushort(__hmul(h, __float2half_rn(-1152.f)))) << 16;
            }
            if (!mbar_wait_warp(&sm.empty[st], ((entry / kStages) & 1) ^ 1, &sm.abort, err)) {
                ok = false;
                break;
            }
            const uint8_t *src = sm.code[cs];
            uint2 c0 = *reinterpret_cast<const uint2 *>(src + in0), c1 = *reinterpret_cast<const uint2 *>(src + in1);
#pragma unroll 1
            for (int i = 0; i < groups; ++i) {
                const uint32_t w = __shfl_sync(0xffffffffu, fg, i);
                const uint32_t nx = 2048 * min(i + 1, 7);
                const uint2 d0 = *reinterpret_cast<const uint2 *>(src + nx + in0), d1 = *reinterpret_cast<const uint2 *>(src + nx + in1);
                const __half2 x = *reinterpret_cast<const __half2 *>(&w);
                const __half2 fx = __low2half2(x), gx = __high2half2(x);
                const uint2 w0 = codes_scaled<E4M3>(c0.x, fx, gx), w1 = codes_scaled<E4M3>(c0.y, fx, gx);
                *reinterpret_cast<uint4 *>(dst + 2048 * i + at0) = make_uint4(w0.x, w0.y, w1.x, w1.y);
                const uint2 w2 = codes_scaled<E4M3>(c1.x, fx, gx), w3 = codes_scaled<E4M3>(c1.y, fx, gx);
                *reinterpret_cast<uint4 *>(dst + 2048 * i + at1) = make_uint4(w2.x, w2.y, w3.x, w3.y);
                c0 = d0;
                c1 = d1;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sm.full[st]);
                mbar_arrive(&sm.code_empty[cs]);
            }
        }
        if (ok)
            tree_done(sm, it);
    }
    // Before leaving on an abort, let the copies already issued land.
    if (ct < 32 && own > 1 && __any_sync(0xffffffffu, *static_cast<volatile int *>(&sm.abort))) {
        volatile int no_abort = 0;
        mbar_wait_warp(&sm.own_full[kv], own & 1, &no_abort, nullptr);
    }
}

// ------------------------------------------------------------ softmax
// Which of a tile's 128 keys a node at depth d keeps (where not all rows keep all).
__device__ __forceinline__ void tree_keep(const TreeArgs &a, const TreeSeg &s, const TreeTile &ti, int d, const uint4 &up,
                                          uint32_t (&keep)[4])
{
    if (ti.flags & kDraft) {
        const uint32_t w[4] = {up.x, up.y, up.z, up.w};
        // which ancestors the head's mode keeps at this node's position
        const bool ssa = s.mode == EA_SSA && d >= a.window, blk = s.mode == EA_BLOCK;
        const int64_t mrow = (static_cast<int64_t>(s.b) * a.Hkv + s.h) * a.nBm + (s.L + d) / EA_TILE;
        for (int c = 0; c < 4; ++c) {
            uint32_t k = (c == 0 ? w[0] : c == 1 ? w[1] : c == 2 ? w[2] : w[3]) & cols_below(s.n, c);
            if (ssa || blk)
                for (uint32_t left = k; left; left &= left - 1) {
                    const int j = 32 * c + __ffs(left) - 1;
                    // the nearest valid depth, as for the node itself: the position stays below L + n, the block
                    // below nBm (tree_unit)
                    const int dj = min(max(a.depth[static_cast<int64_t>(s.b) * a.T + j], 0), s.n - 1), pos = s.L + dj;
                    const bool in = ssa ? pos < a.sink || d - dj < a.window : a.block_mask[mrow * a.nBm + pos / EA_TILE] != 0;
                    if (!in)
                        k &= ~(left & (0u - left));
                }
            keep[0] = c == 0 ? k : keep[0];
            keep[1] = c == 1 ? k : keep[1];
            keep[2] = c == 2 ? k : keep[2];
            keep[3] = c == 3 ? k : keep[3];
        }
    } else {
        const int lim = s.L - ti.key0;
        const bool row_in = s.mode != EA_BLOCK || (ti.flags & ((s.L + d) / EA_TILE > s.L / EA_TILE ? kRow1 : kRow0));
        const int sink = a.sink - ti.key0;                       // columns below are kept,
        const int win = s.L - ti.key0 + d - a.window + 1;        // and those from here on
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            keep[c] = row_in ? cols_below(lim, c) : 0u;
            if (s.mode == EA_SSA)
                keep[c] &= cols_below(sink, c) | ~cols_below(win, c);
        }
    }
}

// -inf where the row does not keep the key.
__device__ __forceinline__ void mask32(uint32_t (&x)[32], uint32_t keep)
{
#pragma unroll
    for (int i = 0; i < 32; ++i)
        x[i] = (keep >> i) & 1u ? x[i] : 0xff800000u;
}

// 8-bit caches: a key's number in S to its logit (cs: what the row's queries stand for, and the call's scale), and
// log2 of what its numbers of V stand for, + 127, which joins it: p = 2^(x unit + v + shift - m) is what multiplies those
// numbers, and p times `inv`, shifted, the softmax's weight.  (Not zero: a masked -inf stays one.)
__device__ __forceinline__ float key_unit(float cs, uint32_t u)
{
    return fmaxf(cs * __uint_as_float(u << 23), 1e-37f);
}

__device__ __forceinline__ float val_log(uint32_t u)
{
    return static_cast<float>(u);
}

__device__ __forceinline__ float val_inv(uint32_t u)
{
    return __uint_as_float((254u - u) << 23);
}

__device__ __forceinline__ float max32(const uint32_t (&x)[32], float m)
{
    float a = m, b = __uint_as_float(x[1]);
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        a = max3f(a, __uint_as_float(x[i]), __uint_as_float(x[i + 2]));
        b = max3f(b, __uint_as_float(x[i + 1]), __uint_as_float(x[i + 3]));
    }
    return fmaxf(a, b);
}

// p = 2^(c x + d) of 32 columns into TMEM as bf16 (f16); the sums of its even and odd ones grow.
template <bool F16>
__device__ __forceinline__ void exp32(const uint32_t (&x)[32], uint64_t c, uint64_t d, uint64_t &sum, uint32_t tp)
{
    uint32_t p[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float e0, e1;
        f2_unpack(f2_fma(f2_pack(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), c, d), e0, e1);
        e0 = ex2(e0);
        e1 = ex2(e1);
        sum = f2_add(sum, f2_pack(e0, e1));
        if constexpr (F16) {
            const __half2 h = __floats2half2_rn(e0, e1);
            p[i] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            p[i] = pack_bf16x2(e0, e1);
        }
    }
    tmem_st16(tp, p);
}

// The same with p in two bf16 parts, the second one in the other half of the columns: a row that keeps few keys takes
// one probability's rounding, 2^-8 of it, almost whole (outputs of values in [2.2, 3.8) over 2 to 500 keys were off by up to
// 0.01 beyond their own rounding).  So do the prefill and the decode, up to the same number.  (256 sequences of 512, trees of 4:
// 140 us without, 177 with; nothing where more keys are kept.)  The first part is cut, not rounded, and the second 2^-23 p more than what is left,
// so that both are positive wherever p is: an infinity among the values stays one.
__device__ __forceinline__ void exp32_parts(const uint32_t (&x)[32], uint64_t c, uint64_t d, uint64_t &sum, uint32_t tp)
{
    uint32_t p[32];
    const uint64_t more = f2_pack(1.f + 0x1p-23f, 1.f + 0x1p-23f);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float e0, e1;
        f2_unpack(f2_fma(f2_pack(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), c, d), e0, e1);
        e0 = ex2(e0);
        e1 = ex2(e1);
        const uint64_t e = f2_pack(e0, e1);
        sum = f2_add(sum, e);
        const uint32_t u0 = __float_as_uint(e0), u1 = __float_as_uint(e1);
        p[i] = __byte_perm(u0, u1, 0x7632);
        f2_unpack(f2_fma(e, more, f2_pack(__uint_as_float((u0 & 0xffff0000u) | 0x80000000u), __uint_as_float((u1 & 0xffff0000u) | 0x80000000u))), e0, e1);
        p[16 + i] = pack_bf16x2(e0, e1);
    }
    tmem_st32(tp, p);
}

// A row's 128 scores go through its thread's registers once (bf16 caches); beside the
// converting warps there is no room for them, they are read from TMEM twice.  The 32 columns'
// P takes the place of the first half of their S.
template <class Smem>
__device__ __forceinline__ void tree_softmax(const TreeArgs &a, Smem &sm, uint32_t tmem, int warp, int lane)
{
    constexpr bool TWO = sizeof(sm.q) > kTBytes;
    const float NEG_INF = -__int_as_float(0x7f800000);
    uint32_t *err = &a.hdr->error;
    const int wg = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_base + 128 * wg, to = tmem + lane_base + kTColO;
    auto place = [&](int c) { return ts + 32 * c; };
    uint32_t own = 0, tile0 = 0, joined = 0;
    const TreeSeg *sp;
    for (uint32_t it = 0; (sp = tree_take(a, sm, it)) != nullptr; ++it) {
        const TreeSeg &s = *sp;
        const bool two = TWO && s.two;
        const int mt = two ? wg : 0, tl = quot(r, a.g, a.inv_g), hh = r - tl * a.g;
        const int t = s.tok0 + mt * a.tpt + tl;
        const bool valid = tl < a.tpt && t < s.n;
        const bool active = __any_sync(0xffffffffu, valid);
        const int64_t node = static_cast<int64_t>(s.b) * a.T + t;
        int d = 0;
        uint4 up = make_uint4(0u, 0u, 0u, 0u);
        if (valid) {
            d = a.depth[node];
            if (s.t1 == s.nt && !s.dead)
                up = a.mask[node];
            if (d < 0 || d >= s.n) {
                raise_error(err, EA_DEVERR_CHECK);
                d = d < 0 ? 0 : s.n - 1;
            }
        }
        // 8-bit caches: the queries as f16, each row times a power of two that puts its largest below
        // 2^11 (exact but for what is 2^-35 of it); `cs` undoes it.  With one M tile the first
        // warpgroup does it and hands cs on.
        float cs = a.scale_log2;
        bool have = true;
        if constexpr (Smem::Q8) {
            if (!mbar_wait_warp(&sm.q_full, it & 1, &sm.abort, err))
                return;
            have = two || wg == 0;
            if (have) {
                if (it > 0 && !mbar_wait_warp(&sm.o_free, (it - 1) & 1, &sm.abort, err))
                    return;                            // (the last range's maxima have been read)
                if (active) {
                    uint8_t *row = sm.q[mt] + r * 128;
                    auto part = [&](int c) { return reinterpret_cast<uint4 *>(row + (c >> 3) * kTHalf + (((c & 7) ^ (r & 7)) << 4)); };
                    float mx[2] = {0.f, 0.f};
#pragma unroll 8
                    for (int c = 0; c < 16; ++c)
                        mx[c & 1] = max_mag(*part(c), mx[c & 1]);
                    mx[0] = fmaxf(mx[0], mx[1]);
                    if (exponent_of(mx[0]) == 255) {
                        mx[0] = 0.f;
#pragma unroll 1
                        for (int c = 0; c < 16; ++c)
                            mx[0] = max_finite(*part(c), mx[0]);
                    }
                    const int e = min(10 + 127 - exponent_of(mx[0]), 120);
                    const float f = pow2f(e);
                    asm volatile("" ::: "memory");       // (read again, not kept)
#pragma unroll 8
                    for (int c = 0; c < 16; ++c)
                        *part(c) = bf16_to_f16(*part(c), f);
                    cs = a.scale_log2 * pow2f(-e);
                }
                if (!two)
                    sm.ml[0][r].x = cs;
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sm.q_ready);
        }
        float m = NEG_INF, l = 0.f;                    // of the exponents' unit: log2
        int steps = 0;
        for (int tt = s.t0 + (two ? 0 : wg); tt < s.t1; tt += two ? 1 : 2, ++own, ++steps) {
            if (!mbar_wait_warp(&sm.s_full[wg], own & 1, &sm.abort, err))
                return;
            if (active) {
                tc_fence_after();
                const uint32_t tile = tile0 + (tt - s.t0);
                const int flags = sm.tile[tile % kTInfos].flags;
                const bool edge = (flags & kEdge) != 0;
                const int chunks = ((flags >> kGroups) + 1) / 2;     // of 32 columns, that hold keys
                uint32_t keep[4];
                bool odd = false;
                const bool wide = Smem::Q8 && (flags & kWide);
                if (edge || wide) {
                    tree_keep(a, s, sm.tile[tile % kTInfos], d, up, keep);
                    if ((flags & kMixed) || wide) {
                        if (!mbar_wait_warp(&sm.ready[tile % kTReady], (tile / kTReady) & 1, &sm.abort, err))
                            return;
                        odd = sm.odd[tile % kTReady] != 0;
                    }
                }
                __syncwarp();
                if constexpr (Smem::Q8) {
                    if (!have)
                        cs = sm.ml[0][r].x;
                    have = true;
                }
                const uint8_t (&units)[2][8] = sm.group_unit[Smem::Q8 ? tile % kTInfos : 0];
                // (O's product of this warpgroup's step before is over: its S is issued behind that.)
                auto grow = [&](float mx) {
                    const bool grew = mx > m + kTGrow;
                    if (__any_sync(0xffffffffu, grew)) {
                        const float f = grew && m != NEG_INF ? ex2(m - mx) : 1.f;
                        m = grew ? mx : m;
                        l *= f;
                        if (steps > 0) {
#pragma unroll 1
                            for (int c = 0; c < 8; ++c) {
                                uint32_t o[16];
                                tmem_ld16(to + 128 * wg + 16 * c, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    asm volatile("" : "+r"(o[i]));
                                    o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                }
                                tmem_st16(to + 128 * wg + 16 * c, o);
                            }
                            tmem_wait_st();
                        }
                    }
                };
                if (Smem::Q8 && !edge && !wide) {
                    // (few registers, and little code: see tree_convert)
                    const uint32_t v0 = units[1][0];
                    const float unit = key_unit(cs, units[0][0]), v = val_log(v0);
                    float mx = NEG_INF;
#pragma unroll 1
                    for (int c = 0; c < 4; c += 2) {
                        uint32_t x[2][32];
                        tmem_ld32(ts + 32 * c, x[0]);
                        tmem_ld32(ts + 32 * c + 32, x[1]);
                        tmem_wait_ld();
                        tie32(x[0]);
                        tie32(x[1]);
                        mx = max32(x[1], max32(x[0], mx));
                    }
                    grow(fmaf(mx, unit, v));
                    const float db = v + kTShift - (m == NEG_INF ? 0.f : m);
                    const uint64_t c2 = f2_pack(unit, unit), d2 = f2_pack(db, db);
                    uint64_t sum = 0;
                    uint32_t x[32], y[32];
                    tmem_ld32(ts + 96, x);
#pragma unroll 1
                    for (int c = 3; c >= 0; --c) {
                        tmem_wait_ld();
                        tie32(x);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            y[i] = x[i];
                        tie32(y);
                        tmem_ld32(ts + 32 * max(c - 1, 0), x);       // the next, under this one's work
                        exp32<true>(y, c2, d2, sum, place(c));
                    }
                    tmem_wait_ld();
                    tie32(x);
                    float p0, p1;
                    f2_unpack(sum, p0, p1);
                    l = fmaf(p0 + p1, val_inv(v0), l);
                } else if (!Smem::Q8 && !edge && !s.few) {
                    float mx = NEG_INF;
                    uint32_t x[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        tmem_ld32(ts + 32 * c, x[c]);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        tie32(x[c]);
                        mx = max32(x[c], mx);
                    }
                    grow(mx * a.scale_log2);
                    const float db = m == NEG_INF ? 0.f : -m;
                    const uint64_t c2 = f2_pack(a.scale_log2, a.scale_log2), d2 = f2_pack(db, db);
                    uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        exp32<false>(x[c], c2, d2, c & 1 ? sum1 : sum0, place(c));
                    float u, v;
                    f2_unpack(f2_add(sum0, sum1), u, v);
                    l += u + v;
                } else if (!odd) {
                    // 32 columns at a time, those that hold keys
                    const float unit = Smem::Q8 ? key_unit(cs, units[0][0]) : a.scale_log2, v = Smem::Q8 ? val_log(units[1][0]) : 0.f;
                    float mx = NEG_INF;
#pragma unroll 1
                    for (int c = 0; c < chunks; ++c) {
                        uint32_t x[32];
                        tmem_ld32(ts + 32 * c, x);
                        tmem_wait_ld();
                        tie32(x);
                        if (Smem::Q8 || edge)
                            mask32(x, c == 0 ? keep[0] : c == 1 ? keep[1] : c == 2 ? keep[2] : keep[3]);
                        mx = max32(x, mx);
                    }
                    grow(fmaf(mx, unit, v));
                    const float db = v + (Smem::Q8 ? kTShift : 0.f) - (m == NEG_INF ? 0.f : m);
                    const uint64_t c2 = f2_pack(unit, unit), d2 = f2_pack(db, db);
                    uint64_t sum = 0;
#pragma unroll 1
                    for (int c = 0; c < chunks; ++c) {
                        uint32_t x[32];
                        tmem_ld32(ts + 32 * c, x);
                        tmem_wait_ld();
                        tie32(x);
                        if (Smem::Q8 || edge)
                            mask32(x, c == 0 ? keep[0] : c == 1 ? keep[1] : c == 2 ? keep[2] : keep[3]);
                        if (!Smem::Q8 && s.few)
                            exp32_parts(x, c2, d2, sum, place(c));
                        else
                            exp32<Smem::Q8>(x, c2, d2, sum, place(c));
                    }
                    float p0, p1;
                    f2_unpack(sum, p0, p1);
                    l = fmaf(p0 + p1, Smem::Q8 ? val_inv(units[1][0]) : 1.f, l);
                } else {
                    // V holds infinities or NaN in a tile that rows keep differently, or keys have units of
                    // their own: the kept ones one by one, so that none reaches a row that does not keep it (the first ones of
                    // a range write O, once nobody reads the last range's)
                    if (steps == 0 && it > 0 && !mbar_wait_warp(&sm.o_free, (it - 1) & 1, &sm.abort, err))
                        return;
                    const uint8_t *v0 = sm.ring[(2 * tile + 1) % Smem::kStages];
                    float mx = NEG_INF, sum = 0.f;
                    // a key's units
                    auto ku = [&](int k) {
                        return !Smem::Q8 ? a.scale_log2 : key_unit(cs, flags & kDraft ? sm.own_unit[it % kTSegs][0][k] : units[0][k >> 4]);
                    };
                    auto vu = [&](int k) -> uint32_t { return flags & kDraft ? sm.own_unit[it % kTSegs][1][k] : units[1][k >> 4]; };
#pragma unroll 1
                    for (int k = 0; k < 16 * (flags >> kGroups); ++k) {
                        uint32_t sk = tmem_ld1(ts + k);
                        tmem_wait_ld();
                        asm volatile("" : "+r"(sk));
                        const uint32_t kw = k < 32 ? keep[0] : k < 64 ? keep[1] : k < 96 ? keep[2] : keep[3];
                        mx = (kw >> (k & 31)) & 1u ? fmaxf(mx, fmaf(__uint_as_float(sk), ku(k), Smem::Q8 ? val_log(vu(k)) : 0.f)) : mx;
                    }
                    grow(mx);
                    const float db = (Smem::Q8 ? kTShift : 0.f) - (m == NEG_INF ? 0.f : m);
#pragma unroll 1
                    for (int dc = 0; dc < 8; ++dc) {              // 16 dims at a time
                        uint32_t raw[16];
                        float o[16];
                        if (steps > 0) {
                            tmem_ld16(to + 128 * wg + 16 * dc, raw);
                            tmem_wait_ld();
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            asm volatile("" : "+r"(raw[i]));
                            o[i] = steps > 0 ? __uint_as_float(raw[i]) : 0.f;
                        }
#pragma unroll 1
                        for (int k = 0; k < 16 * (flags >> kGroups); ++k) {
                            __syncwarp();
                            uint32_t sk = tmem_ld1(ts + k);
                            tmem_wait_ld();
                            asm volatile("" : "+r"(sk));
                            const uint32_t kw = k < 32 ? keep[0] : k < 64 ? keep[1] : k < 96 ? keep[2] : keep[3];
                            if ((kw >> (k & 31)) & 1u) {
                                const float p = ex2(fmaf(__uint_as_float(sk), ku(k), (Smem::Q8 ? val_log(vu(k)) : 0.f) + db));
                                sum += dc > 0 ? 0.f : Smem::Q8 ? p * val_inv(vu(k)) : p;
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    const uint4 v = *reinterpret_cast<const uint4 *>(
                                        v0 + (dc >> 2) * kTHalf + k * 128 + ((((dc & 3) * 2 + j) ^ (k & 7)) << 4));
                                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                    for (int q = 0; q < 4; ++q) {
                                        const float2 x = Smem::Q8 ? f16_f32(w[q])
                                                                  : make_float2(__uint_as_float(w[q] << 16),
                                                                                __uint_as_float(w[q] & 0xffff0000u));
                                        o[8 * j + 2 * q] = fmaf(p, x.x, o[8 * j + 2 * q]);
                                        o[8 * j + 2 * q + 1] = fmaf(p, x.y, o[8 * j + 2 * q + 1]);
                                    }
                                }
                            }
                        }
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            raw[i] = __float_as_uint(o[i]);
                        tmem_st16(to + 128 * wg + 16 * dc, raw);
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
        float M = m;
        if (!two) {
            float2 x0 = make_float2(M, l), x1 = x0;
            if constexpr (Smem::Q8) {
                // (one place a row, there is no room for two: the second warpgroup's, then the first's)
                if (wg == 0) {
                    if (!mbar_wait_warp(&sm.ml_full[0], joined & 1, &sm.abort, err))
                        return;
                    x1 = sm.ml[0][r];
                    sm.ml[0][r] = x0;
                } else {
                    sm.ml[0][r] = x1;
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sm.ml_full[wg ^ 1]);
                if (wg == 1) {
                    if (!mbar_wait_warp(&sm.ml_full[1], joined & 1, &sm.abort, err))
                        return;
                    x0 = sm.ml[0][r];
                }
            } else {
                sm.ml[wg][r] = x0;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sm.ml_full[0]);
                if (!mbar_wait_warp(&sm.ml_full[0], joined & 1, &sm.abort, err))
                    return;
                x0 = sm.ml[0][r];
                x1 = sm.ml[1][r];
            }
            ++joined;
            M = fmaxf(x0.x, x1.x);
            // 1 where nothing but NaN (or no key) was met, so that a NaN stays
            f0 = x0.x == NEG_INF ? 1.f : ex2(x0.x - M);
            f1 = x1.x == NEG_INF ? 1.f : ex2(x1.x - M);
            both = s.t1 - s.t0 > 1;
            l = both ? x0.y * f0 + x1.y * f1 : x0.y * f0;
        }
        if (active) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const bool none = l == 0.f, whole = s.t0 == 0 && s.t1 == s.nt;
            f0 *= inv;
            f1 *= inv;
            const int64_t prow = static_cast<int64_t>(s.slot) * a.rows_slot + mt * kTTile + r;
            const int c0 = two ? 0 : 2 * wg, c1 = two ? 4 : c0 + 2;
            __nv_bfloat16 *o = a.O + s.b * a.o_sb + t * a.o_st + (s.h * a.g + hh) * a.o_sh;
            float *po = a.part_o + prow * EA_HEAD_DIM;
            const uint32_t t0 = to + (two ? 128 * wg : 0);
#pragma unroll 1
            for (int c = c0; c < c1; ++c) {
                uint32_t x[32];
                __syncwarp();
                tmem_ld32(t0 + 32 * c, x);
                if (both) {
                    uint32_t y[32];
                    tmem_ld32(to + 128 + 32 * c, y);
                    tmem_wait_ld();
                    tie32(x);
                    tie32(y);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        x[i] = __float_as_uint(fmaf(__uint_as_float(y[i]), f1, __uint_as_float(x[i]) * f0));
                } else {
                    tmem_wait_ld();
                    tie32(x);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        x[i] = __float_as_uint(__uint_as_float(x[i]) * f0);
                }
                if (none) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        x[i] = 0u;
                }
                if (valid) {
                    if (whole) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t w[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                w[k] = pack_bf16x2(__uint_as_float(x[8 * i + 2 * k]), __uint_as_float(x[8 * i + 2 * k + 1]));
                            reinterpret_cast<uint4 *>(o + 32 * c)[i] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    } else if (in_bounds(prow, 2 * static_cast<int64_t>(gridDim.x) * a.rows_slot, err)) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            st_global_v8(po + 32 * c + 8 * i, x + 8 * i);
                    }
                }
            }
            if (valid && (two || wg == 0)) {
                const float l2 = none ? NEG_INF : (M == NEG_INF ? 0.f : M) - (Smem::Q8 ? kTShift + 127.f : 0.f) + tree_lg2(l);
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
        tree_done(sm, it);
    }
}

// ------------------------------------------------------------ kernels
// A barrier a lane and step, by its place among them.
template <class Smem>
__device__ __forceinline__ void tree_barriers(Smem &sm, int lane)
{
    constexpr int S = Smem::kStages, C = Smem::kCodes, users = 8 + 3 + (Smem::Q8 ? kTConvWarps : 0);
    struct Kind {
        int n, count;
    };
    constexpr Kind kinds[] = {
        {S, Smem::Q8 ? kTConvWarps / 2 : 1},            // full
        {S, 2},                                         // empty: the product that used it, and the warp that looks V over
        {C, 1}, {C, kTConvWarps / 2},                   // code_full, code_empty
        {kTReady, 1},
        {kTSegs, 1}, {kTSegs, users},
        {1, 1}, {1, 1},                                 // q_full, q_empty
        {2, 1}, {2, 4}, {2, 1},                         // s_full, p_full, o_done
        {1, 1}, {2, Smem::Q8 ? 4 : 8}, {1, 8}, {1, 2},  // seg_done, ml_full, o_free, drain
        {1, 8}, {2, 1}, {2, 4},                         // q_ready, own_full, own_max
    };
    constexpr int kAll = static_cast<int>((offsetof(Smem, seg) - offsetof(Smem, full)) / sizeof(uint64_t));
    static_assert(2 * S + 2 * C + kTReady + 2 * kTSegs + 2 + 6 + 5 + 5 == kAll, "every barrier is set up");
    for (int i = lane; i < kAll; i += 32) {
        int count = 1, end = 0;
#pragma unroll
        for (int k = 0; k < static_cast<int>(sizeof(kinds) / sizeof(Kind)); ++k) {
            count = i >= end ? kinds[k].count : count;
            end += kinds[k].n;
        }
        mbar_init(sm.full + i, count);
    }
    if (lane == 0)
        sm.abort = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    __syncwarp();
}

template <int FMT, bool TWO>
__global__ void __launch_bounds__(FMT == EA_CACHE_BF16 ? kTThreads : kTThreadsQ8, 1)
    tree_attn_kernel(const __grid_constant__ TreeMaps tm, const TreeArgs a)
{
    constexpr bool kQ8 = FMT != EA_CACHE_BF16;
    using Smem = TreeSmem<kQ8, TWO>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (smem_u32(smem_raw) & 1023u) {                  // the operands' layout needs it
        if (threadIdx.x == 0)
            raise_error(&a.hdr->error, EA_DEVERR_BOUNDS);
        return;
    }
    // The producer sets the barriers up and goes on to its range and its first copies; the others wait
    // for that and for TMEM.
    if (warp == kTProducerWarp) {
        tree_barriers(sm, lane);
        if (a.B * a.Hkv <= kTWarpUnits) {
            griddep_wait();
            named_bar_arrive(1, blockDim.x);
            tree_range(a, sm, lane, 1);
            __syncwarp();
        }
    }
    if (warp == kTQkWarp) {
        tmem_alloc(&sm.tmem_base, 512);
        tmem_relinquish();
    }
    if (a.B * a.Hkv > kTWarpUnits) {
        griddep_wait();
        tree_range(a, sm, threadIdx.x, blockDim.x / 32);
        tc_fence_before();
        __syncthreads();
    } else if (warp != kTProducerWarp) {
        griddep_wait();
        tc_fence_before();
        named_bar_sync(1, blockDim.x);
    }
    griddep_launch_dependents();
    tc_fence_after();
    const uint32_t tmem = warp == kTProducerWarp ? 0u : sm.tmem_base;

    // Registers go to the softmax: 256 x 208 + 128 x 88 of the launch's 384 x 168, or, with
    // converting warps, 256 x 128 + 128 x 72 + 256 x 72 of its 640 x 96.
    if (warp < 8) {
        if constexpr (kQ8)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
        else
            asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        tree_softmax(a, sm, tmem, warp, lane);
    } else if (warp < kTConvWarp) {
        if constexpr (kQ8)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        else
            asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == kTProducerWarp) {
            tree_producer(tm, a, sm, lane);
        } else if (warp == kTQkWarp) {
            tree_qk(a, sm, tmem);
        } else if (warp == kTPvWarp) {
            tree_pv(a, sm, tmem);
        } else {
            tree_fix(tm, a, sm, lane);
        }
    } else {
        if constexpr (kQ8) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
            tree_convert<FMT == EA_CACHE_E4M3>(tm, a, sm, (warp - kTConvWarp) / 4, threadIdx.x % 128, lane);
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kTQkWarp) {
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
    // eight parts' weights and data at a time
    float M = NEG_INF, w = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int cb = c0; cb <= c1; cb += 8) {
        float l[8];
        float4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int64_t p = part(min(cb + k, c1));
            l[k] = cb + k <= c1 ? a.part_lse[p] : NEG_INF;
            x[k] = *reinterpret_cast<const float4 *>(a.part_o + p * EA_HEAD_DIM + 4 * lane);
        }
        float mx = M;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            mx = fmaxf(mx, l[k]);
        const float f = M == NEG_INF ? 1.f : ex2(M - mx);            // (nothing, or NaN, before)
        M = mx;
        const float ref = M == NEG_INF ? 0.f : M;
        w *= f;
        acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float e = cb + k <= c1 ? ex2(l[k] - ref) : 0.f;
            if (cb + k <= c1) {
                w += e;
                acc.x = fmaf(e, x[k].x, acc.x);
                acc.y = fmaf(e, x[k].y, acc.y);
                acc.z = fmaf(e, x[k].z, acc.z);
                acc.w = fmaf(e, x[k].w, acc.w);
            }
        }
    }
    const float ref = M == NEG_INF ? 0.f : M;
    const float inv = w == 0.f ? 0.f : 1.f / w;
    const uint2 o = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    *reinterpret_cast<uint2 *>(a.O + b * a.o_sb + t * a.o_st + qh * a.o_sh + 4 * lane) = o;
    if (a.LSE && lane == 0)
        a.LSE[(static_cast<int64_t>(b) * a.Hq + qh) * a.T + t] =
            (w == 0.f ? NEG_INF : ref + tree_lg2(w)) * 0.69314718055994531f;
}

// ------------------------------------------------------------ host
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

// The tiles of a step at most, which the kernel counts in 32 bits.
static bool tree_tiles_ok(int B, int Hkv, int pairs, int Lmax)
{
    return static_cast<double>(B) * Hkv * pairs * (ceil_div(Lmax, kTTile) + 1 + kTPartTiles) < 2147483648.;
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

template <int FMT, bool TWO>
static cudaError_t launch_tree(const TreeMaps &tm, const TreeArgs &a, int grid, bool after, cudaStream_t st, int dev)
{
    constexpr size_t kSmem = sizeof(TreeSmem<FMT != EA_CACHE_BF16, TWO>);
    static bool attr_done[64] = {};   // the attribute is set once per device
    if (dev >= 64 || !attr_done[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(tree_attn_kernel<FMT, TWO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(kSmem));
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
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = after ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, tree_attn_kernel<FMT, TWO>, tm, a);
}

template <int FMT>
static cudaError_t launch_tree_fmt(const TreeMaps &tm, const TreeArgs &a, int grid, bool after, cudaStream_t st, int dev)
{
    return a.rows_slot > kTTile ? launch_tree<FMT, true>(tm, a, grid, after, st, dev)
                                : launch_tree<FMT, false>(tm, a, grid, after, st, dev);
}

} // namespace ea

using namespace ea;

extern "C" size_t ea_tree_workspace_size(int B, int T, int Hq, int Hkv, int d, int Lmax)
{
    if (!tree_sizes_ok(B, T, Hq, Hkv, d) || Lmax < 1)
        return 0;
    const TreeWs w = tree_ws_layout(B, T, Hq, Hkv, Lmax);
    return tree_tiles_ok(B, Hkv, w.pairs, Lmax) ? w.total : 0;
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
    if (!tree_tiles_ok(B, Hkv, w.pairs, Lmax))
        return EA_ERR_UNSUPPORTED;
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
        const int box = a.box128 ? kTTile : 64;
        if (!encode_tmap_u8_plain(&tm.k, a.c.code[0], Hkv, a.c.rows, a.c.outer, cache->kv_str, box) ||
            !encode_tmap_u8_plain(&tm.v, a.c.code[1], Hkv, a.c.rows, a.c.outer, cache->kv_str, box))
            return EA_ERR_INVALID_ARG;
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
    // positions stay below 2^31 - 128: larger limits say the same (and the window's first column, less 96, stays in 32 bits)
    a.sink = sink < (1 << 30) ? sink : 0x7fffffff;
    a.window = window < 0x7fffffff - 128 ? window : 0x7fffffff - 128;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.inv_Hkv = 1.f / static_cast<float>(Hkv);
    a.inv_g = 1.f / static_cast<float>(a.g);
    a.inv_tpt = 1.f / static_cast<float>(a.tpt);
    a.page_log2 = -1;
    for (int k = 6; k < 31; ++k)
        if (a.c.rows == 1 << k)
            a.page_log2 = k;

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
        e = launch_tree_fmt<EA_CACHE_BF16>(tm, a, grid, block_mask != nullptr, st, dev);
    else if (a.c.format == EA_CACHE_E4M3)
        e = launch_tree_fmt<EA_CACHE_E4M3>(tm, a, grid, block_mask != nullptr, st, dev);
    else
        e = launch_tree_fmt<EA_CACHE_INT8>(tm, a, grid, block_mask != nullptr, st, dev);
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
