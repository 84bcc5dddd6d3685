// ea_decode_plan.cuh - the work decomposition of a decode step, shared by the
// bf16 and the 8-bit decode: which keys a (b, KV head) unit keeps, how they are
// cut into chunks, and where a chunk's 64-key tiles lie.
#pragma once

#include "ea_device.cuh"

namespace ea {

constexpr int kDecKeys = 64;                           // keys per tile
constexpr int kSplitBits = 11;                         // chunk code: unit << 11 | split

struct DecodeArgs {
    const __nv_bfloat16 *q;
    int64_t q_sb, q_sh;
    const int32_t *seqlens;
    const uint8_t *m;
    int32_t *unit_first;
    int32_t *unit_splits;
    int32_t *chunks;
    float *part_o;
    float *part_lse;
    ea_ws_header *hdr;
    __nv_bfloat16 *O;
    int64_t o_sb, o_sh;
    float *LSE;
    int B, Hq, Hkv, g, Lmax, sink, window, num_splits, max_splits, num_sms;
    float scale_log2;
    // block-sparse heads: mask [B][Hkv][nBm][nBm] (NULL when no head may be
    // EA_BLOCK) and, per unit, the kept blocks of its decode row
    const uint8_t *block_mask;
    int nBm;
    int32_t *blk_count;
    uint16_t *blk_list;
    // paged cache (page_size == 0: one contiguous [B][Lmax] cache)
    const int32_t *block_table;
    int64_t bt_stride;
    int page_size, num_pages;
    // a single sequence (B * Hkv <= kSelfPlanUnits): every split CTA plans the
    // step itself and takes chunks blockIdx.x + k * gridDim.x, with no planner
    // launch and no queue
    int self_plan;
    int chunk_min, chunk_max;   // automatic chunk size (kept keys)
    int whole_waves;            // the chunks are to fill whole waves of the SMs (see Waves)
    int64_t max_chunks;         // chunks that the workspace has room for
};

// Up to this many units a step is planned inside the split kernel.  Measured
// per step against the planner launch: B = 1 x 8 KV heads 36.9 -> 35.3 us; at
// B = 4 and 8 the fixed chunk assignment balances worse than the queue (+1.4 %,
// +4.6 %), so larger batches keep the planner.
constexpr int kSelfPlanUnits = 8;

// The plan of a self-planned step, in shared memory.
struct SelfPlan {
    int first[kSelfPlanUnits], ns[kSelfPlanUnits], total;
};

// Kept keys of one (b, KV head) unit as at most two contiguous ranges:
// visited index v < n0 is key v, v >= n0 is key w0 + (v - n0).  A BLOCK unit
// (blk >= 0 kept blocks) is walked as 64-key tiles instead: two per kept
// block, the last block cut at L (see block_tiles).
struct KeySegs {
    int n;
    int n0;
    int w0;
    int blk;      // kept blocks of a BLOCK unit, -1 otherwise
    int L;
};

__device__ __forceinline__ bool unit_keys(const DecodeArgs &a, int b, int h, KeySegs &ks)
{
    int L = a.seqlens[b];
    const int mode = a.m[b * a.Hkv + h];
    bool ok = true;
    if (L < 0 || L > a.Lmax || mode > EA_BLOCK || (mode == EA_BLOCK && !a.block_mask)) {
        ok = false;
        L = 0;
    }
    ks.L = L;
    ks.blk = -1;
    if (mode == EA_BLOCK && ok) {
        ks.blk = a.blk_count[b * a.Hkv + h];
        ks.n0 = ks.w0 = ks.n = 0;
        return true;
    }
    if (mode == EA_SSA) {
        const int ns = a.sink < L ? a.sink : L;
        const int ws = (L - a.window) > ns ? (L - a.window) : ns;
        ks.n0 = ns;
        ks.w0 = ws;
        ks.n = ns + (L - ws);
    } else {
        ks.n0 = L;
        ks.w0 = L;
        ks.n = L;
    }
    return ok;
}

// Paged cache: the unit's 64-key-aligned tiles are [0, TA) (covering the
// sink) followed by [TB, TL) (covering the window, from the first tile not
// already visited), TL = ceil(L / 64).  Returns the tile count.
__device__ __forceinline__ int paged_tiles(const KeySegs &ks, int &TA, int &TB)
{
    const int L = ks.w0 + (ks.n - ks.n0);
    TA = (ks.n0 + kDecKeys - 1) / kDecKeys;
    const int TL = (L + kDecKeys - 1) / kDecKeys;
    TB = max(ks.w0 / kDecKeys, TA);
    return TA + max(TL - TB, 0);
}

// 64-key tiles of a BLOCK unit: two per kept block, except that the query's
// own block (kept or not, the last one listed when kept) only reaches L.
__device__ __forceinline__ int block_tiles(const DecodeArgs &a, int u, const KeySegs &ks)
{
    if (ks.blk <= 0)
        return 0;
    const int last = a.blk_list[static_cast<int64_t>(u) * a.nBm + ks.blk - 1];
    const int tail = ks.L - last * EA_TILE;          // keys of the last block below L
    return 2 * (ks.blk - 1) + (tail >= EA_TILE ? 2 : (tail + kDecKeys - 1) / kDecKeys);
}

// Kept keys of a unit as the split kernel walks them (whole tiles for a paged
// cache or a BLOCK unit).
__device__ __forceinline__ int unit_work(const DecodeArgs &a, int u, bool &ok)
{
    KeySegs ks;
    ok = unit_keys(a, u / a.Hkv, u % a.Hkv, ks);
    if (ks.blk >= 0)
        return block_tiles(a, u, ks) * kDecKeys;
    int TA, TB;
    return a.page_size ? paged_tiles(ks, TA, TB) * kDecKeys : ks.n;
}

// One CTA per unit: the key blocks kept in the unit's decode row of the block
// mask (row (L - 1) / 128, blocks 0 .. (L - 1) / 128), ascending.  Each pass
// covers 1024 blocks: thread t tests blocks 4t .. 4t + 3 (independent loads),
// and a block-wide exclusive scan of the counts places them.
constexpr int kBlkThreads = 256;

static __global__ void __launch_bounds__(kBlkThreads) decode_blocks_kernel(DecodeArgs a)
{
    __shared__ int warp_tot[kBlkThreads / 32];
    const int u = blockIdx.x, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int b = u / a.Hkv, h = u % a.Hkv;
    const int L = a.seqlens[b];
    griddep_launch_dependents();
    int count = 0;
    if (a.m[u] == EA_BLOCK && L > 0 && L <= a.Lmax) {
        const int qb = (L - 1) / EA_TILE;
        const uint8_t *row = a.block_mask + ((static_cast<int64_t>(b) * a.Hkv + h) * a.nBm + qb) * a.nBm;
        uint16_t *list = a.blk_list + static_cast<int64_t>(u) * a.nBm;
        for (int k0 = 0; k0 <= qb; k0 += 4 * kBlkThreads) {
            uint32_t bits = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int kb = k0 + 4 * tid + j;
                bits |= (kb <= qb && in_bounds(kb, a.nBm, &a.hdr->error) && row[kb] != 0) ? (1u << j)
                                                                                         : 0u;
            }
            const int mine = __popc(bits);
            int incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o)
                    incl += v;
            }
            if (lane == 31)
                warp_tot[warp] = incl;
            __syncthreads();
            int before = 0, total = 0;
#pragma unroll
            for (int w = 0; w < kBlkThreads / 32; ++w) {
                before += w < warp ? warp_tot[w] : 0;
                total += warp_tot[w];
            }
            int pos = count + before + incl - mine;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (((bits >> j) & 1u) && in_bounds(pos, a.nBm, &a.hdr->error))
                    list[pos++] = static_cast<uint16_t>(k0 + 4 * tid + j);
            count += total;
            __syncthreads();   // warp_tot is rewritten by the next pass
        }
    }
    if (tid == 0)
        a.blk_count[u] = count;
}

// Kept keys per chunk when the split count is automatic: about four chunks per SM
// over the step, between chunk_min and chunk_max keys.
__device__ __forceinline__ long long chunk_keys(const DecodeArgs &a, long long work)
{
    const long long sms = a.num_sms > 0 ? a.num_sms : 1;
    const long long target = 4 * sms;
    const long long chunk = (work + target - 1) / target;
    return chunk < a.chunk_min ? a.chunk_min : (chunk > a.chunk_max ? a.chunk_max : chunk);
}

// The same for a step whose chunks are to fill whole waves: one or two per SM in a
// step of fewer than 2048 or 4096 keys per SM, else four, or as many as chunk_max
// takes.  As each unit rounds its chunks up, candidate i of kWaveTries is i eighths
// longer than the work over that number, and the first with no more chunks than it
// is taken, else the last.  (Nine sequences of 30000 keys, full heads: 98.6 -> 92.8
// us; nine ragged ones 50.0 -> 47.4, with streaming heads among them 33.9 -> 30.4.
// The least chunk is work / (4 SMs) or that of chunk_max in whole waves: a step has
// at most 4 SMs + units + units * longest / chunk_max.)
constexpr int kWaveTries = 8;

struct Waves {
    long long target;
    int chunk;               // candidate 0
    __device__ __forceinline__ int candidate(const DecodeArgs &a, int i) const
    {
        const long long c = chunk + static_cast<long long>(chunk) * i / kWaveTries;
        return static_cast<int>(c < a.chunk_max ? c : a.chunk_max);
    }
};

__device__ __forceinline__ Waves waves(const DecodeArgs &a, long long work)
{
    const int sms = a.num_sms > 0 ? a.num_sms : 1;
    // (fp32 quotients, rounded up by one: 64-bit divisions cost the planner 1 us)
    const float each = static_cast<float>(work) / static_cast<float>(sms);
    const int per = each < 2048.f ? 1 : each < 4096.f ? 2 : max(4, static_cast<int>(each / a.chunk_max) + 1);
    Waves w;
    w.target = static_cast<long long>(sms) * per;
    w.chunk = max(static_cast<int>(each / per) + 1, a.chunk_min);
    return w;
}

// Chunks of a unit that count: a short rest runs beside the others.
__device__ __forceinline__ int unit_chunks(int work, int chunk)
{
    return 4ll * work > chunk ? (work + chunk - 1) / chunk : 0;
}

// One CTA: per-unit chunk counts, their prefix sum, and the chunk list.  The
// automatic chunk size aims at about four chunks per SM over the whole step
// (fewer, longer chunks mean fewer partial results to write and merge), between
// a.chunk_min and a.chunk_max kept keys, so that a small
// batch still spreads over every SM.
constexpr int kPlanThreads = 256;
static_assert(kPlanThreads / 32 == kWaveTries, "a warp counts the chunks of one candidate");

static __global__ void __launch_bounds__(kPlanThreads) decode_plan_kernel(DecodeArgs a)
{
    __shared__ long long red_work[kPlanThreads / 32];
    __shared__ int red_chunks[kPlanThreads / 32];
    griddep_launch_dependents();   // the split kernel may start its prologue
    griddep_wait();                // decode_blocks_kernel's lists, where it ran
    const int units = a.B * a.Hkv;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int per = (units + kPlanThreads - 1) / kPlanThreads;
    const int lo = min(tid * per, units), hi = min(lo + per, units);
    // each unit's work, kept in unit_splits until its split count replaces it
    long long mine = 0;
    bool bad = false;
    for (int u = lo; u < hi; ++u) {
        bool ok;
        const int work = unit_work(a, u, ok);
        bad |= !ok;
        a.unit_splits[u] = work;
        mine += work;
    }
    if (bad)
        raise_error(&a.hdr->error, EA_DEVERR_CHECK);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        mine += __shfl_down_sync(0xffffffffu, mine, o);
    if (lane == 0)
        red_work[warp] = mine;
    __syncthreads();
    long long total_work = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w)
        total_work += red_work[w];
    long long chunk;
    if (a.whole_waves) {
        // warp i counts the chunks of candidate i (the units' work is in unit_splits:
        // the barrier above ordered its stores)
        const Waves wv = waves(a, total_work);
        const int c = wv.candidate(a, warp);
        int n = 0;
        if (units <= 32 * kPlanThreads)
            for (int u = lane; u < units; u += 32)
                n += unit_chunks(a.unit_splits[u], c);
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0)
            red_chunks[warp] = n;
        __syncthreads();
        int i = 0;
        while (i < kWaveTries - 1 && red_chunks[i] > wv.target)
            ++i;
        chunk = wv.candidate(a, i);
        __syncthreads();                      // red_chunks is written again
    } else {
        chunk = chunk_keys(a, total_work);
    }
    int local = 0;
    for (int u = lo; u < hi; ++u) {
        const int work = a.unit_splits[u];
        int ns = a.num_splits > 0 ? a.num_splits : static_cast<int>((work + chunk - 1) / chunk);
        ns = ns < 1 ? 1 : (ns > a.max_splits ? a.max_splits : ns);
        a.unit_splits[u] = ns;
        local += ns;
    }
    // exclusive scan of the per-thread chunk counts: lanes, then warps
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += v;
    }
    if (lane == 31)
        red_chunks[warp] = incl;
    __syncthreads();
    int base = 0, grand = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        base += w < warp ? red_chunks[w] : 0;
        grand += red_chunks[w];
    }
    int run = base + incl - local;
    for (int u = lo; u < hi; ++u) {
        a.unit_first[u] = run;
        const int ns = a.unit_splits[u];
        for (int sp = 0; sp < ns; ++sp)
            if (in_bounds(static_cast<int64_t>(run) + sp,
                          a.max_chunks, &a.hdr->error))
                a.chunks[run + sp] = (u << kSplitBits) | sp;
        run += ns;
    }
    if (tid == 0) {
        // (chunks that the list has no room for have been reported)
        a.hdr->n_items = static_cast<uint32_t>(min(static_cast<int64_t>(grand), a.max_chunks));
        a.hdr->work_counter = 0;   // the split kernel's chunk queue
    }
}

// Position of chunk c in the key stream.  Contiguous cache: visited keys
// [v_begin, v_end) in tiles that start at any key.  Paged cache: the unit's
// aligned tiles [v_begin, v_end) (tile indices), tile v at key
// 64 * (v < TA ? v : TB + v - TA).  BLOCK unit (either cache): aligned tiles
// [v_begin, v_end), tile v at key 128 * list[v / 2] + 64 * (v % 2).
struct ChunkInfo {
    int b, h, v_begin, v_end;
    int kept;                 // the unit's kept keys (whole tiles of a BLOCK unit)
    KeySegs ks;
    int a_tiles, b_begin, n_tiles;
    int TA, TB;
    const uint16_t *list;     // BLOCK unit: its kept blocks (NULL otherwise)
};

__device__ __forceinline__ ChunkInfo chunk_info(const DecodeArgs &a, int c, const SelfPlan &plan)
{
    ChunkInfo ci;
    int u, sp, ns;
    if (a.self_plan) {
        // the last unit whose first chunk is <= c (every unit has one chunk at least)
        int lo = 0, hi = a.B * a.Hkv - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (plan.first[mid] <= c)
                lo = mid;
            else
                hi = mid - 1;
        }
        u = lo;
        sp = c - plan.first[u];
        ns = plan.ns[u];
    } else {
        const int code = a.chunks[c];
        u = code >> kSplitBits;
        sp = code & ((1 << kSplitBits) - 1);
        ns = a.unit_splits[u];
    }
    ci.b = u / a.Hkv;
    ci.h = u % a.Hkv;
    unit_keys(a, ci.b, ci.h, ci.ks);
    ci.list = nullptr;
    ci.kept = ci.ks.n;
    if (ci.ks.blk >= 0) {
        ci.list = a.blk_list + static_cast<int64_t>(u) * a.nBm;
        const int nt = block_tiles(a, u, ci.ks);
        ci.kept = nt * kDecKeys;
        const int len = (nt + ns - 1) / ns;
        ci.v_begin = min(sp * len, nt);
        ci.v_end = min(ci.v_begin + len, nt);
        ci.n_tiles = ci.v_end - ci.v_begin;
        ci.a_tiles = ci.b_begin = ci.TA = ci.TB = 0;
        return ci;
    }
    if (a.page_size) {
        const int nt = paged_tiles(ci.ks, ci.TA, ci.TB);
        const int len = (nt + ns - 1) / ns;
        ci.v_begin = min(sp * len, nt);
        ci.v_end = min(ci.v_begin + len, nt);
        ci.n_tiles = ci.v_end - ci.v_begin;
        ci.a_tiles = 0;
        ci.b_begin = 0;
        return ci;
    }
    ci.TA = ci.TB = 0;
    const int len = (ci.ks.n + ns - 1) / ns;
    ci.v_begin = min(sp * len, ci.ks.n);
    ci.v_end = min(ci.v_begin + len, ci.ks.n);
    const int a_end = min(ci.v_end, ci.ks.n0);
    ci.a_tiles = ci.v_begin < a_end ? (a_end - ci.v_begin + kDecKeys - 1) / kDecKeys : 0;
    ci.b_begin = max(ci.v_begin, ci.ks.n0);
    ci.n_tiles = ci.a_tiles + (ci.b_begin < ci.v_end ? (ci.v_end - ci.b_begin + kDecKeys - 1) / kDecKeys : 0);
    return ci;
}

// First key and number of leading keys that may be valid of tile t of a chunk
// (contiguous cache: a tile never straddles the sink and window ranges, and
// all nvalid keys are kept; paged cache: an aligned tile of 64 keys, each
// tested against the kept ranges by the caller).
__device__ __forceinline__ void tile_rows(const DecodeArgs &a, const ChunkInfo &ci, int t,
                                          int &key0, int &nvalid)
{
    if (ci.list) {
        const int v = ci.v_begin + t;
        key0 = EA_TILE * ci.list[v >> 1] + kDecKeys * (v & 1);
        nvalid = min(kDecKeys, ci.ks.L - key0);
        return;
    }
    if (a.page_size) {
        const int v = ci.v_begin + t;
        key0 = kDecKeys * (v < ci.TA ? v : ci.TB + (v - ci.TA));
        nvalid = kDecKeys;
        return;
    }
    if (t < ci.a_tiles) {
        const int v = ci.v_begin + t * kDecKeys;
        key0 = v;
        nvalid = min(kDecKeys, min(ci.v_end, ci.ks.n0) - v);
    } else {
        const int v = ci.b_begin + (t - ci.a_tiles) * kDecKeys;
        key0 = ci.ks.w0 + (v - ci.ks.n0);
        nvalid = min(kDecKeys, ci.v_end - v);
    }
}

// A self-planned step (B * Hkv <= kSelfPlanUnits): warp 0 of every split CTA
// computes the plan decode_plan_kernel would (the same chunk size, split
// counts and chunk order, unit by unit), lane l taking units 2l and 2l + 1, into
// shared memory; CTA 0 also stores each unit's first chunk and split count for
// the merge kernel.
__device__ __forceinline__ void self_plan(const DecodeArgs &a, SelfPlan &plan, int lane)
{
    const int units = a.B * a.Hkv;
    int w[2] = {0, 0};
    bool bad = false;
    long long mine = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int u = 2 * lane + k;
        if (u < units) {
            bool ok;
            w[k] = unit_work(a, u, ok);
            bad |= !ok;
            mine += w[k];
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        mine += __shfl_xor_sync(0xffffffffu, mine, o);
    long long chunk;
    if (a.whole_waves) {
        // few units: room for each one's last chunk
        const Waves wv = waves(a, mine);
        const float t = static_cast<float>(wv.target);
        chunk = min(static_cast<int>(wv.chunk * (t / (t - min(static_cast<float>(units), t / 2.f)))) + 1,
                    a.chunk_max);
    } else {
        chunk = chunk_keys(a, mine);
    }
    int ns[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (2 * lane + k < units) {
            int n = a.num_splits > 0 ? a.num_splits : static_cast<int>((w[k] + chunk - 1) / chunk);
            ns[k] = n < 1 ? 1 : (n > a.max_splits ? a.max_splits : n);
        }
    const int local = ns[0] + ns[1];
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += v;
    }
    int first = incl - local;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int u = 2 * lane + k;
        if (u < units) {
            plan.first[u] = first;
            plan.ns[u] = ns[k];
            if (blockIdx.x == 0) {
                a.unit_first[u] = first;
                a.unit_splits[u] = ns[k];
            }
        }
        first += ns[k];
    }
    if (lane == 31)
        plan.total = incl;
    if (bad && blockIdx.x == 0)
        raise_error(&a.hdr->error, EA_DEVERR_CHECK);
}

} // namespace ea
