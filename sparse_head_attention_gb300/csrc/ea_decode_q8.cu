// ea_decode_q8.cu - one decode step over a KV cache held in 8 bits with a scale
// per block of tokens and KV head, and the attention weight each key received.
//
// With codes c and scales s, a key's logit is x_j = scale * s^K_j (q . c^K_j) and
// the output O = sum_j p_j s^V_j c^V_j, p = softmax(x).  The scales act on whole
// keys, so the products run on the codes, and s^K joins the logit and s^V the
// probability: w_j = 2^(x_j log2 e + log2 s^V_j - M), with M the running maximum
// of that exponent, is what multiplies c^V, and the normaliser is
// l = sum_j w_j / s^V_j.
//
// A step reads each kept key's 256 bytes once and is bound by HBM: at the
// measured 6.79 TB/s an SM receives 45 bytes a ns, one 64-key tile of K and V
// (16 KB) every 0.37 us.
//   - The producer warp keeps kQ8Stages tiles in flight by TMA (one 128-byte
//     swizzled box of 64 rows per K or V); its own time per tile counts (700 cycles
//     at that rate), so its lanes work out 32 tiles' places at once, and the
//     compute warps load the scales themselves, a tile ahead.  (Scales as 4-byte
//     asynchronous copies on the tile's barrier: 434 us for 16 sequences of
//     64K; written beside the tile by the producer: 385.)
//   - The compute warps take whole tiles in turn (tile n goes to warp n mod
//     kQ8Warps): no exchange between warps within a chunk of keys, the softmax's
//     maximum is reduced once per 64 keys, and a warp has several tile times for
//     the latency of its own tile.
//   - Joining warps add the compute warps' results of a chunk up while those are
//     at the next chunk, so that a chunk's end waits for nobody (nine ragged
//     sequences of all head kinds 40.4 -> 37.6 us with key weights, nine of up to
//     30000 keys and full heads 57 -> 51; with one such warp instead of four the
//     end of a short step is its: one sequence of 32K 14.4 us, not 13.6).
//   - Products are m16n8k16 f16 MMAs with the keys (then the head dims) as the 16
//     rows and the group's up to eight query heads as the 8 columns, so no row is
//     padding: S^T = C^K Q^T and O^T += C^V^T W^T.  e4m3 and int8 codes are exact
//     in f16; Q (bf16) is exact in f16 after a power of two per row, down to
//     2^-24 of the row's largest element; w is scaled to at most 2^14, so f16
//     keeps 11 bits of every w above 2^-28 of the largest and 2^-38 of it as the
//     last step.  Accumulators, maxima, sums and partial results are fp32.
//   - One 8x8 b16 matrix of ldmatrix holds 16 codes of each of 8 rows, so a lane
//     gets 4 neighbouring codes: for S^T that is one k16 step of its row once Q's
//     columns are taken in the same order; for V^T the transposed load gives 2
//     dims of 2 keys, which pair up by key.
// Chunks (runs of one unit's tiles, taken from a queue), their planning and the
// masks are those of the bf16 decode (ea_decode_plan.cuh) with all tiles 64-key
// aligned.  (One equal range of all units' tiles per SM instead leaves no SM idle,
// but neighbouring heads' rows, neighbours in memory, are then no longer read at
// the same time: 333 -> 371 us for 16 sequences of 64K.)  A merge joins the chunks
// of each (sequence, head), and with key weights a last kernel turns the stored
// logits into exp(x - LSE) and sums them over the group.
//
// Measured: 16 sequences of 64K, 8 KV heads, 317 - 333 us on different GPUs of
// the kind (2.15 GB: 0.95 - 1.0 of the measured HBM rate); one of 32K with two full
// and six streaming heads 13.6 us (20 MB, bound by the latency of a plan, a chunk
// of nine tiles, two joins and a second launch).
#include <cuda.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "ea_cache.cuh"
#include "ea_decode_plan.cuh"
#include "ea_internal.h"

namespace ea {

constexpr int kQ8Stages = 12;
constexpr int kQ8TileBytes = kDecKeys * EA_HEAD_DIM;   // K or V codes of one tile: 8 KB
constexpr int kQ8Warps = 6;                            // compute warps
constexpr int kQ8Joiners = 4;                          // warps that add the compute warps' results up
constexpr int kQ8Threads = (kQ8Warps + 1 + kQ8Joiners) * 32;   // + one producer warp
constexpr int kQ8Groups = kDecKeys / 16;               // 16-key groups of a tile: one scale each at most
constexpr float kQ8Shift = 14.f;                       // w <= 2^14

struct __align__(1024) Q8Smem {
    uint8_t k[kQ8Stages][kQ8TileBytes];
    uint8_t v[kQ8Stages][kQ8TileBytes];
    float red_o[kQ8Warps][8][EA_HEAD_DIM];
    float red_m[kQ8Warps][8];
    float red_l[kQ8Warps][8];
    uint64_t full[kQ8Stages];
    uint64_t empty[kQ8Stages];
    uint64_t chunk_full[2], chunk_empty[2];
    uint64_t red_full, red_empty;             // the warps' results of a chunk
    int chunk[2];
    int abort;
    SelfPlan plan;
};
constexpr size_t kQ8SmemBytes = sizeof(Q8Smem) + 1024;
static_assert(kQ8SmemBytes <= 232448, "shared memory of one CTA");
// Every use of a stage belongs to the same warp, which so waits for its uses in
// order.  (A wait names a phase by its parity: were tile n - kQ8Stages another
// warp's, a warp early at tile n could take the phase before it, still being
// loaded, for its own.)
static_assert(kQ8Stages % kQ8Warps == 0, "a stage belongs to one warp");

struct Q8Args {
    DecodeArgs d;
    const float *ks, *vs;     // [outer][Hkv][nsb]
    int nsb, log2sb;
    float *scores;            // log2-domain logits [unit][Lmax][gp], or NULL
    float *lse2;              // final log2 LSE [B * Hq]
    float *key_w;             // [unit][Lmax]
    int gp, accumulate;
};

__device__ __forceinline__ void q8_ldsm_x4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ void q8_ldsm_x4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ uint32_t movmatrix_t(uint32_t a)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                 "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ float lg2(float x)
{
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ bool key_kept(const KeySegs &ks, int key)
{
    return (key < ks.n0 || key >= ks.w0) && key < ks.L;
}

template <bool E4M3, bool WEIGHTS>
__global__ void __launch_bounds__(kQ8Threads, 1)
    decode_q8_kernel(const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const Q8Args qa)
{
    extern __shared__ uint8_t smem_raw[];
    Q8Smem &sm = *reinterpret_cast<Q8Smem *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const DecodeArgs &a = qa.d;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int r = lane >> 2, qd = lane & 3;
    const float NEG_INF = -__int_as_float(0x7f800000);
    volatile int *abort = &sm.abort;

    if (tid == 0) {
        sm.abort = 0;
        for (int s = 0; s < kQ8Stages; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sm.chunk_full[s], 1);
            mbar_init(&sm.chunk_empty[s], kQ8Warps + kQ8Joiners);
        }
        mbar_init(&sm.red_full, kQ8Warps);
        mbar_init(&sm.red_empty, kQ8Joiners);
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    __syncthreads();
    if (a.self_plan) {
        if (warp == 0)
            self_plan(a, sm.plan, lane);
        __syncthreads();
    }
    griddep_wait();
    griddep_launch_dependents();
    const int total = a.self_plan ? sm.plan.total : static_cast<int>(a.hdr->n_items);

    if (warp == kQ8Warps) {
        // ------------------------------------------------------------ producer
        uint32_t issued = 0, phase = 0;
        int st = 0;                             // issued % kQ8Stages, and its phase
        bool ok = true;
        for (int it = 0; ok; ++it) {
            const int slot = it & 1;
            if (!mbar_wait_warp(&sm.chunk_empty[slot], ((it >> 1) & 1) ^ 1, abort, &a.hdr->error))
                break;
            int c = -1;
            if (lane == 0) {
                const uint32_t x = a.self_plan ? blockIdx.x + static_cast<uint32_t>(it) * gridDim.x
                                               : atomicAdd(&a.hdr->work_counter, 1u);
                c = x < static_cast<uint32_t>(total) ? static_cast<int>(x) : -1;
                sm.chunk[slot] = c;
                mbar_arrive(&sm.chunk_full[slot]);
            }
            c = __shfl_sync(0xffffffffu, c, 0);
            if (c < 0)
                break;
            const ChunkInfo ci = chunk_info(a, c, sm.plan);
            // Lane j holds the place of tile 32 k + j (row, and sequence or page),
            // looked up a group of 32 tiles ahead of the copies that need it.
            int row_of = 0, outer_of = 0, row_next = 0, outer_next = 0;
            auto place = [&](int t, int &row, int &outer) {
                row = 0;
                outer = ci.b;
                if (t >= ci.n_tiles)
                    return;
                int key0, nv;
                tile_rows(a, ci, t, key0, nv);
                row = key0;
                if (a.block_table) {
                    const int at = key0 / a.page_size;
                    row = key0 - at * a.page_size;
                    outer = in_bounds(at, a.Lmax / a.page_size, &a.hdr->error)
                                ? a.block_table[ci.b * a.bt_stride + at]
                                : -1;
                    // a page outside the cache is reported; its copy reads the
                    // fill value (a box outside the tensor is zero-filled)
                    if (outer < 0 || outer >= a.num_pages) {
                        raise_error(&a.hdr->error, EA_DEVERR_CHECK);
                        outer = -1;
                    }
                }
            };
            place(lane, row_next, outer_next);
            for (int t = 0; t < ci.n_tiles; ++t) {
                if ((t & 31) == 0) {
                    row_of = row_next;
                    outer_of = outer_next;
                    place(t + 32 + lane, row_next, outer_next);
                }
                const int row = __shfl_sync(0xffffffffu, row_of, t & 31);
                const int outer = __shfl_sync(0xffffffffu, outer_of, t & 31);
                if (!mbar_wait_warp(&sm.empty[st], phase ^ 1, abort, &a.hdr->error)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(&sm.full[st], 2 * kQ8TileBytes);
                    tma_load_4d(sm.k[st], &tm_k, 0, ci.h, row, outer, &sm.full[st]);
                    tma_load_4d(sm.v[st], &tm_v, 0, ci.h, row, outer, &sm.full[st]);
                }
                __syncwarp();
                ++issued;
                if (++st == kQ8Stages) {
                    st = 0;
                    phase ^= 1;
                }
            }
        }
        // Before leaving on an abort, let the copies already issued land.
        if (__any_sync(0xffffffffu, *abort)) {
            for (uint32_t k = issued > kQ8Stages ? issued - kQ8Stages : 0; k < issued; ++k) {
                volatile int no_abort = 0;
                mbar_wait_warp(&sm.full[k % kQ8Stages], (k / kQ8Stages) & 1, &no_abort, nullptr);
            }
        }
        return;
    }

    // The compute warps and the joining warps: chunk number `it` (-1: none left).
    auto next_chunk = [&](int it) {
        const int slot = it & 1;
        const bool ok = mbar_wait_warp(&sm.chunk_full[slot], (it >> 1) & 1, abort, &a.hdr->error);
        const int c = ok ? sm.chunk[slot] : -1;
        __syncwarp();
        if (ok && lane == 0)
            mbar_arrive(&sm.chunk_empty[slot]);
        return c;
    };

    if (warp > kQ8Warps) {
        // ------------------------------------------------------------ joining warps
        // add up the compute warps' results of a chunk while they go on to the next
        for (int it = 0;; ++it) {
            const int c = next_chunk(it);
            if (c < 0 || !mbar_wait_warp(&sm.red_full, it & 1, abort, &a.hdr->error))
                return;
            for (int hh = warp - kQ8Warps - 1; hh < a.g; hh += kQ8Joiners) {
                float M = NEG_INF;
#pragma unroll
                for (int w = 0; w < kQ8Warps; ++w)
                    M = fmaxf(M, sm.red_m[w][hh]);
                float lsum = 0.f;
                float4 osum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kQ8Warps; ++w) {
                    const float mw = sm.red_m[w][hh];
                    // 1 where nothing but NaN (or no key) was met, so that a NaN stays
                    const float f = mw == NEG_INF ? 1.f : ex2(mw - M);
                    const float4 x = *reinterpret_cast<const float4 *>(&sm.red_o[w][hh][4 * lane]);
                    lsum = fmaf(sm.red_l[w][hh], f, lsum);
                    osum.x = fmaf(x.x, f, osum.x);
                    osum.y = fmaf(x.y, f, osum.y);
                    osum.z = fmaf(x.z, f, osum.z);
                    osum.w = fmaf(x.w, f, osum.w);
                }
                const int64_t pidx = static_cast<int64_t>(c) * a.g + hh;
                if (!in_bounds(pidx, a.max_chunks * a.g, &a.hdr->error))
                    continue;
                if (lsum == 0.f)
                    osum = make_float4(0.f, 0.f, 0.f, 0.f);
                else
                    osum = make_float4(osum.x / lsum, osum.y / lsum, osum.z / lsum, osum.w / lsum);
                *reinterpret_cast<float4 *>(a.part_o + pidx * EA_HEAD_DIM + 4 * lane) = osum;
                const float Mb = (M == NEG_INF ? 0.f : M) - kQ8Shift;
                if (lane == 0)
                    a.part_lse[pidx] = lsum == 0.f ? NEG_INF : Mb + lg2(lsum);
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sm.red_empty);
        }
    }

    // ---------------------------------------------------------------- compute
    uint32_t base = 0;                          // tiles of the chunks before this one
    for (int it = 0;; ++it) {
        const int c = next_chunk(it);
        if (c < 0)
            return;
        bool ok = true;
        const ChunkInfo ci = chunk_info(a, c, sm.plan);
        // Q as the B operand: column n = head r of the group (heads >= g are
        // zero), k = 2q.. and 2q + 8.. are dims 16 j + 4 q .. + 3; times a power
        // of two that puts the row's largest element in [2^10, 2^11)
        uint32_t qb[8][2];
        float cs[2];                            // log2-domain logit per unit of the product, heads 2 qd, 2 qd + 1
        {
            const bool real = r < a.g;
            const __nv_bfloat16 *qrow = a.q + ci.b * a.q_sb + (ci.h * a.g + (real ? r : 0)) * a.q_sh;
            uint2 raw[8];
            uint32_t mx = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                raw[j] = make_uint2(0u, 0u);
                if (real)
                    raw[j] = *reinterpret_cast<const uint2 *>(qrow + 16 * j + 4 * qd);
                mx = max(mx, max(max(raw[j].x & 0x7fffu, (raw[j].x >> 16) & 0x7fffu),
                                 max(raw[j].y & 0x7fffu, (raw[j].y >> 16) & 0x7fffu)));
            }
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            int e = 10 + 127 - static_cast<int>(mx >> 7);        // an infinity or a NaN stays one
            e = mx >= 0x7f80u ? 0 : e < -126 ? -126 : e > 120 ? 120 : e;
            const float f = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                qb[j][0] = pack_f16x2(__uint_as_float(raw[j].x << 16) * f,
                                      __uint_as_float(raw[j].x & 0xffff0000u) * f);
                qb[j][1] = pack_f16x2(__uint_as_float(raw[j].y << 16) * f,
                                      __uint_as_float(raw[j].y & 0xffff0000u) * f);
            }
            const float inv = a.scale_log2 / f;
            cs[0] = __shfl_sync(0xffffffffu, inv, 8 * qd);       // lane of head 2 qd
            cs[1] = __shfl_sync(0xffffffffu, inv, 8 * qd + 4);
        }
        float o[8][4];
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[n][e] = 0.f;
        float m_run[2] = {NEG_INF, NEG_INF}, l_part[2] = {0.f, 0.f};
        float *score = nullptr;
        if constexpr (WEIGHTS)
            score = qa.scores + (static_cast<int64_t>(ci.b) * a.Hkv + ci.h) * a.Lmax * qa.gp + 2 * qd;

        // sc: lane i < 8 holds K's (then V's) scale of group i % 4
        auto tile = [&](auto masked_tag, int s, int key0, float sc) {
            constexpr bool kMasked = decltype(masked_tag)::value;
            const uint32_t kb = smem_u32(sm.k[s]), vb = smem_u32(sm.v[s]);
            const int lrow = ((lane >> 3) & 1) * 8 + (lane & 7), lcol = lane >> 4;
            bool keep[2 * kQ8Groups];            // keys r and r + 8 of each group
            if constexpr (kMasked) {
#pragma unroll
                for (int i = 0; i < 2 * kQ8Groups; ++i) {
                    const int key = key0 + 8 * i + r;
                    keep[i] = ci.list ? key < ci.ks.L : key_kept(ci.ks, key);
                }
            }
            // S^T: 16 keys x 8 heads per group
            float x[kQ8Groups][4];
#pragma unroll
            for (int i = 0; i < kQ8Groups; ++i) {
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
                const int row = 16 * i + lrow;
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    uint32_t w[4], f[4];
                    q8_ldsm_x4(kb + row * 128 + (((j + lcol) ^ (row & 7)) << 4), w);
                    codes_f16<E4M3, false>(w[0], f[0], f[2]);
                    codes_f16<E4M3, false>(w[1], f[1], f[3]);
                    mma_f16(acc, f, qb[j][0], qb[j][1]);
                    codes_f16<E4M3, false>(w[2], f[0], f[2]);
                    codes_f16<E4M3, false>(w[3], f[1], f[3]);
                    mma_f16(acc, f, qb[j + 1][0], qb[j + 1][1]);
                }
                const float ks = __shfl_sync(0xffffffffu, sc, i);
                const float lv = lg2(__shfl_sync(0xffffffffu, sc, kQ8Groups + i));
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[i][e] = __fmul_rn(acc[e], cs[e & 1] * ks);   // not fused with lv: as it is stored
                if constexpr (WEIGHTS) {
                    if (2 * qd < qa.gp) {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (!kMasked || keep[2 * i + e]) {
                                float *p = score + static_cast<int64_t>(key0 + 16 * i + 8 * e + r) * qa.gp;
                                if (qa.gp == 1)
                                    *p = x[i][2 * e];
                                else
                                    *reinterpret_cast<float2 *>(p) = make_float2(x[i][2 * e], x[i][2 * e + 1]);
                            }
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[i][e] += lv;
                    if (kMasked && !keep[2 * i + (e >> 1)])
                        x[i][e] = NEG_INF;
                }
            }
            // online softmax: the maximum over the tile of each of the two heads
            bool grew = false;
            float m_new[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = m_run[e];
#pragma unroll
                for (int i = 0; i < kQ8Groups; ++i)
                    mx = max3f(mx, x[i][e], x[i][e + 2]);
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                m_new[e] = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                grew |= m_new[e] > m_run[e];
            }
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float f = m_run[e] == NEG_INF ? 0.f : ex2(m_run[e] - m_new[e]);
                    l_part[e] *= f;
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
                        o[n][e] *= f;
                        o[n][e + 2] *= f;
                    }
                    m_run[e] = m_new[e];
                }
            }
            const float mb[2] = {(m_run[0] == NEG_INF ? 0.f : m_run[0]) - kQ8Shift,
                                 (m_run[1] == NEG_INF ? 0.f : m_run[1]) - kQ8Shift};
#pragma unroll
            for (int i = 0; i < kQ8Groups; ++i) {
                const float iv = __frcp_rn(__shfl_sync(0xffffffffu, sc, kQ8Groups + i));
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[i][e] = ex2(x[i][e] - mb[e & 1]);
                    if (!kMasked || keep[2 * i + (e >> 1)])
                        l_part[e & 1] = fmaf(x[i][e], iv, l_part[e & 1]);
                }
                // W^T of the group: keys as k, heads as n
                const uint32_t b0 = movmatrix_t(pack_f16x2(x[i][0], x[i][1]));
                const uint32_t b1 = movmatrix_t(pack_f16x2(x[i][2], x[i][3]));
                uint32_t z0 = 0xffffffffu, z1 = 0xffffffffu;     // V's bytes of the keys 2 qd, 2 qd + 1 (+ 8)
                if constexpr (kMasked) {
                    const int k0 = key0 + 16 * i + 2 * qd;
                    auto half = [&](int key) { return ci.list ? key < ci.ks.L : key_kept(ci.ks, key); };
                    z0 = (half(k0) ? 0xffffu : 0u) | (half(k0 + 1) ? 0xffff0000u : 0u);
                    z1 = (half(k0 + 8) ? 0xffffu : 0u) | (half(k0 + 9) ? 0xffff0000u : 0u);
                }
                const int row = 16 * i + lrow;
#pragma unroll
                for (int n = 0; n < 8; n += 2) {
                    uint32_t w[4], f[4];
                    q8_ldsm_x4_t(vb + row * 128 + (((n + lcol) ^ (row & 7)) << 4), w);
                    if constexpr (kMasked) {
                        w[0] &= z0;
                        w[1] &= z1;
                        w[2] &= z0;
                        w[3] &= z1;
                    }
                    codes_f16<E4M3, true>(w[0], f[0], f[1]);
                    codes_f16<E4M3, true>(w[1], f[2], f[3]);
                    mma_f16(o[n], f, b0, b1);
                    codes_f16<E4M3, true>(w[2], f[0], f[1]);
                    codes_f16<E4M3, true>(w[3], f[2], f[3]);
                    mma_f16(o[n + 1], f, b0, b1);
                }
            }
        };

        // Lanes 0 - 3: K's scales of a tile's 16-key groups, 4 - 7: V's; 1 for groups
        // that begin behind the sequence's end (their blocks may hold nothing)
        // and for pages outside the cache (their codes read as zeros).
        auto load_scale = [&](int t) -> float {
            if (lane >= 2 * kQ8Groups || t >= ci.n_tiles)
                return 1.f;
            int key0, nv;
            tile_rows(a, ci, t, key0, nv);
            int row = key0 + 16 * (lane % kQ8Groups), outer = ci.b;
            if (row >= ci.ks.L)
                return 1.f;
            if (a.block_table) {
                const int at = key0 / a.page_size;
                row -= at * a.page_size;
                outer = in_bounds(at, a.Lmax / a.page_size, &a.hdr->error)
                            ? a.block_table[ci.b * a.bt_stride + at]
                            : -1;
                if (outer < 0 || outer >= a.num_pages)
                    return 1.f;
            }
            const float *p = lane < kQ8Groups ? qa.ks : qa.vs;
            return __ldg(p + (static_cast<int64_t>(outer) * a.Hkv + ci.h) * qa.nsb + (row >> qa.log2sb));
        };
        // this warp's tiles of the chunk
        const int first = static_cast<int>((warp + kQ8Warps - base % kQ8Warps) % kQ8Warps);
        float sc_next = load_scale(first);
        for (int t = first; ok && t < ci.n_tiles; t += kQ8Warps) {
            const float sc = sc_next;
            sc_next = load_scale(t + kQ8Warps);
            const uint32_t n = base + t;
            const int s = n % kQ8Stages;
            if (!mbar_wait_warp(&sm.full[s], (n / kQ8Stages) & 1, abort, &a.hdr->error)) {
                ok = false;
                break;
            }
            int key0, nv;
            tile_rows(a, ci, t, key0, nv);
            const int last = key0 + kDecKeys;
            const bool whole = ci.list ? last <= ci.ks.L
                                       : last <= ci.ks.n0 || (key0 >= ci.ks.w0 && last <= ci.ks.L);
            if (whole)
                tile(std::false_type{}, s, key0, sc);
            else
                tile(std::true_type{}, s, key0, sc);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sm.empty[s]);
        }
        base += ci.n_tiles;

        // this warp's results -> shared memory, once those of the chunk before have
        // been joined.  They are placed by the chunk's tiles that they hold (first,
        // first + kQ8Warps, ...): which warp that is depends on the chunks its CTA took
        // before, and the order of the sums must not.
        if (!ok || !mbar_wait_warp(&sm.red_empty, (it & 1) ^ 1, abort, &a.hdr->error))
            return;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l_part[e] += __shfl_xor_sync(0xffffffffu, l_part[e], 4);
            l_part[e] += __shfl_xor_sync(0xffffffffu, l_part[e], 8);
            l_part[e] += __shfl_xor_sync(0xffffffffu, l_part[e], 16);
            const int head = 2 * qd + e;
            if (head < a.g) {
#pragma unroll
                for (int n = 0; n < 8; ++n)
                    *reinterpret_cast<float2 *>(&sm.red_o[first][head][16 * n + 2 * r]) =
                        make_float2(o[n][e], o[n][e + 2]);
                if (r == 0) {
                    sm.red_m[first][head] = m_run[e];
                    sm.red_l[first][head] = l_part[e];
                }
            }
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&sm.red_full);
    }
}

// ---------------------------------------------------------------- merge
// One CTA per (b, q head): joins the unit's chunks (partial O and log2 LSE) by
// their weights 2^(lse - max).  A NaN partial makes the result NaN.  Groups of
// 128 threads take a share of the chunks each, eight chunks' loads at a time.
// Bound by latency: 4.5 us for 288 rows of up to twelve chunks (cold).
constexpr int kQ8MergeGroups = 4;

__global__ void __launch_bounds__(kQ8MergeGroups * EA_HEAD_DIM, 2) decode_q8_merge_kernel(const Q8Args qa)
{
    __shared__ float gm[kQ8MergeGroups], gw[kQ8MergeGroups];
    __shared__ float go[kQ8MergeGroups][EA_HEAD_DIM];
    const DecodeArgs &a = qa.d;
    const float NEG_INF = -__int_as_float(0x7f800000);
    const int b = blockIdx.x, qh = blockIdx.y;
    const int dd = threadIdx.x % EA_HEAD_DIM, grp = threadIdx.x / EA_HEAD_DIM;
    griddep_wait();
    griddep_launch_dependents();
    const int u = b * a.Hkv + qh / a.g, hh = qh % a.g;
    const int first = a.unit_first[u];
    int ns = a.unit_splits[u];
    if (!in_bounds(static_cast<int64_t>(first) + ns - 1, a.max_chunks, &a.hdr->error))
        ns = 0;
    const int64_t base = static_cast<int64_t>(first) * a.g + hh;
    const int groups = blockDim.x / EA_HEAD_DIM;
    const int per = (ns + groups - 1) / groups;
    const int s0 = min(grp * per, ns), s1 = min(s0 + per, ns);
    float m = NEG_INF, w = 0.f, osum = 0.f;
    for (int s = s0; s < s1; s += 8) {
        float l[8], o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const bool in = s + k < s1;
            const int64_t pidx = base + static_cast<int64_t>(in ? s + k : s) * a.g;
            l[k] = in ? a.part_lse[pidx] : NEG_INF;
            o[k] = in ? a.part_o[pidx * EA_HEAD_DIM + dd] : 0.f;
        }
        float mb = m;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            mb = fmaxf(mb, l[k]);
        const float f = m == NEG_INF ? 1.f : ex2(m - mb);      // (nothing, or NaN, before)
        w *= f;
        osum *= f;
        m = mb;
        const float ref = m == NEG_INF ? 0.f : m;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float e = ex2(l[k] - ref);                   // an empty chunk: 0, its o too
            w += e;
            osum = fmaf(e, o[k], osum);
        }
    }
    if (dd == 0) {
        gm[grp] = m;
        gw[grp] = w;
    }
    go[grp][dd] = osum;
    __syncthreads();
    if (grp == 0) {
        float M = NEG_INF;
#pragma unroll
        for (int k = 0; k < kQ8MergeGroups; ++k)
            if (k < groups)
                M = fmaxf(M, gm[k]);
        float wsum = 0.f, o = 0.f;
#pragma unroll
        for (int k = 0; k < kQ8MergeGroups; ++k)
            if (k < groups) {
                const float f = gm[k] == NEG_INF ? 1.f : ex2(gm[k] - M);
                wsum = fmaf(gw[k], f, wsum);
                o = fmaf(go[k][dd], f, o);
            }
        const float ref = M == NEG_INF ? 0.f : M;
        a.O[b * a.o_sb + qh * a.o_sh + dd] = __float2bfloat16_rn(wsum == 0.f ? 0.f : o / wsum);
        if (dd == 0) {
            const float l2 = wsum == 0.f ? NEG_INF : ref + lg2(wsum);
            if (qa.lse2)
                qa.lse2[static_cast<int64_t>(b) * a.Hq + qh] = l2;
            if (a.LSE)
                a.LSE[static_cast<int64_t>(b) * a.Hq + qh] = l2 * 0.69314718055994531f;
        }
    }
}

// ---------------------------------------------------------------- key weights
// key_w[unit][j] (+)= sum over the group's heads of 2^(logit - lse) for the kept
// keys j of the unit, 0 for the others below its length.  A thread per key, its
// group's logits side by side.  They come from L2, where the split kernel left them:
// 0.87M keys of 72 units, four heads each, 7.3 us (13.9 MB read).
constexpr int kQ8WThreads = 256;
constexpr int kQ8WKeys = 4 * kQ8WThreads;

__global__ void __launch_bounds__(kQ8WThreads) decode_q8_weights_kernel(const Q8Args qa)
{
    const DecodeArgs &a = qa.d;
    griddep_wait();
    const int u = blockIdx.y, b = u / a.Hkv, h = u % a.Hkv;
    const int L = a.seqlens[b];
    const int j0 = blockIdx.x * kQ8WKeys;
    if (L < 0 || L > a.Lmax || j0 >= L)
        return;
    KeySegs ks;
    unit_keys(a, b, h, ks);
    const uint8_t *row = nullptr;
    if (ks.blk >= 0)
        row = a.block_mask + (static_cast<int64_t>(u) * a.nBm + (L - 1) / EA_TILE) * a.nBm;
    float lse[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        lse[e] = e < a.g ? qa.lse2[static_cast<int64_t>(b) * a.Hq + h * a.g + e] : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = j0 + i * kQ8WThreads + threadIdx.x;
        if (j >= L)
            break;
        const bool kept = row ? row[j / EA_TILE] != 0 : key_kept(ks, j);
        const int64_t at = static_cast<int64_t>(u) * a.Lmax + j;
        float w = 0.f;
        if (kept) {
            const float *p = qa.scores + at * qa.gp;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < a.g)
                    w += ex2(p[e] - lse[e]);
        }
        qa.key_w[at] = qa.accumulate ? qa.key_w[at] + w : w;
    }
}

// ---------------------------------------------------------------- host
// Keys per chunk when the split count is automatic (see Waves).  Measured on one
// sequence of 32K with two full and six streaming heads: chunks of 2048 keys 19.3
// us, one chunk per SM 13.6.
constexpr int kQ8MinChunk = 256;
constexpr int kQ8MaxChunk = 8192;
constexpr int kQ8Sms = 152;                  // the plan is for this GPU: a workspace's size depends on it
constexpr int kQ8MaxSplits = 1024;
constexpr int kQ8MaxSplitKeys = 1 << 24;     // a chunk's joining warps wait for all of it, 2 s at most

// Chunks of a step at most: the caller's count per unit, or four per SM (or, in a
// step too long for that, one per kQ8MaxChunk keys), one more for every unit's
// remainder.
static int64_t q8_max_chunks(int64_t units, int Lmax, int num_splits)
{
    if (num_splits > 0)
        return units * num_splits;
    const int64_t longest = ceil_div(Lmax, EA_TILE) * EA_TILE;     // whole tiles
    const int64_t per_unit = ceil_div(longest, kQ8MinChunk) < kQ8MaxSplits ? ceil_div(longest, kQ8MinChunk)
                                                                          : kQ8MaxSplits;
    const int64_t n = 4 * kQ8Sms + units + units * ceil_div(longest, kQ8MaxChunk);
    return n < units * per_unit ? n : units * per_unit;
}

struct Q8Ws {
    DecodeWs d;
    size_t lse2, scores, total;
    int64_t max_chunks;
    int gp;
};

static Q8Ws q8_ws_layout(int B, int Hq, int Hkv, int Lmax, int num_splits, bool weights)
{
    Q8Ws w{};
    const size_t units = static_cast<size_t>(B) * Hkv;
    const int g = Hq / Hkv;
    w.max_chunks = q8_max_chunks(static_cast<int64_t>(units), Lmax, num_splits);
    const size_t chunks = static_cast<size_t>(w.max_chunks);
    size_t off = sizeof(ea_ws_header);
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align_up(off + bytes, 256);
        return at;
    };
    w.d.unit_first = take(sizeof(int32_t) * units);
    w.d.unit_splits = take(sizeof(int32_t) * units);
    w.d.chunks = take(sizeof(int32_t) * chunks);
    w.d.partial_o = take(sizeof(float) * chunks * g * EA_HEAD_DIM);
    w.d.partial_lse = take(sizeof(float) * chunks * g);
    w.d.blk_count = take(sizeof(int32_t) * units);
    w.d.blk_list = take(sizeof(uint16_t) * units * static_cast<size_t>(ceil_div(Lmax, EA_TILE)));
    w.gp = g == 1 ? 1 : g == 2 ? 2 : g <= 4 ? 4 : g <= 6 ? 6 : 8;
    w.lse2 = take(sizeof(float) * static_cast<size_t>(B) * Hq);
    w.scores = off;
    if (weights)
        take(sizeof(float) * units * Lmax * w.gp);
    w.total = off;
    return w;
}

// A kernel that starts its prologue under the end of the call's one before it.
template <typename A>
static cudaError_t launch_q8_after(void (*kernel)(A), const A &a, dim3 grid, int threads, cudaStream_t st)
{
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <bool E4M3, bool WEIGHTS>
static cudaError_t launch_q8(const CUtensorMap &tk, const CUtensorMap &tv, const Q8Args &a, int grid,
                             cudaStream_t st, int dev)
{
    static bool attr_done[64] = {};   // the attribute is set once per device
    if (dev >= 64 || !attr_done[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(decode_q8_kernel<E4M3, WEIGHTS>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(kQ8SmemBytes));
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
    cfg.blockDim = dim3(kQ8Threads);
    cfg.dynamicSmemBytes = kQ8SmemBytes;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = a.d.self_plan ? 0 : 1;
    return cudaLaunchKernelEx(&cfg, decode_q8_kernel<E4M3, WEIGHTS>, tk, tv, a);
}

// A decode of many (b, head) rows joins each row's few chunks with one group of
// 128 threads; few rows take four groups each.
static cudaError_t launch_q8_merge(const Q8Args &a, cudaStream_t st)
{
    const int groups = static_cast<int64_t>(a.d.B) * a.d.Hq >= 2ll * a.d.num_sms ? 1 : kQ8MergeGroups;
    return launch_q8_after(decode_q8_merge_kernel, a, dim3(a.d.B, a.d.Hq), groups * EA_HEAD_DIM, st);
}

} // namespace ea

using namespace ea;

extern "C" size_t ea_decode_q8_workspace_size(int B, int Hq, int Hkv, int d, int Lmax, int num_splits,
                                              int with_weights)
{
    if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq / Hkv > 8 || d != EA_HEAD_DIM || Lmax < 1 ||
        num_splits < 0 || num_splits > 1024)
        return 0;
    return q8_ws_layout(B, Hq, Hkv, Lmax, num_splits, with_weights != 0).total;
}

extern "C" ea_status ea_hybrid_attn_decode_q8(const void *q, const ea_cache *cache, void *O, float *LSE,
                                              const int64_t q_str[3], const int64_t o_str[3],
                                              const int32_t *seqlens, int B, int Hq, float scale,
                                              const uint8_t *m, int sink, int window,
                                              const uint8_t *block_mask, int block_size,
                                              int num_splits, float *key_weights, int accumulate,
                                              void *workspace, size_t ws_bytes, void *stream)
{
    if (!q || !O || !q_str || !o_str || !seqlens || !m)
        return EA_ERR_INVALID_ARG;
    CacheDev c;
    ea_status why;
    if (!cache_dev(cache, B, c, why))
        return why;
    const int Hkv = c.Hkv, Lmax = c.cap;
    if (Hq < 1 || Hq % Hkv != 0 || sink < 0 || window < 1 || !(scale > 0.f) || num_splits < 0 ||
        num_splits > 1024 || block_size != EA_TILE)
        return EA_ERR_INVALID_ARG;
    const int64_t nBm = ceil_div(Lmax, EA_TILE);
    if (c.format == EA_CACHE_BF16 || Hq / Hkv > 8 || (block_mask && nBm > 65535) ||
        (c.table && c.rows % kDecKeys) ||
        (num_splits > 0 && ceil_div(Lmax, num_splits) > kQ8MaxSplitKeys))
        return EA_ERR_UNSUPPORTED;
    if (q_str[2] != 1 || o_str[2] != 1 || q_str[0] <= 0 || q_str[1] <= 0 || o_str[0] <= 0 ||
        o_str[1] <= 0 || q_str[0] % 8 || q_str[1] % 8)
        return EA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(O)) & 15u)
        return EA_ERR_INVALID_ARG;
    if (Hq > 65535 || static_cast<int64_t>(B) * Hkv >= (int64_t(1) << (31 - kSplitBits)) ||
        q8_max_chunks(static_cast<int64_t>(B) * Hkv, Lmax, num_splits) >= (int64_t(1) << 31) ||
        (key_weights && static_cast<int64_t>(B) * Hkv > 65535))
        return EA_ERR_UNSUPPORTED;
    const Q8Ws L = q8_ws_layout(B, Hq, Hkv, Lmax, num_splits, key_weights != nullptr);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || ws_bytes < L.total)
        return EA_ERR_WORKSPACE;

    alignas(64) CUtensorMap tk, tv;
    if (!encode_tmap_u8_4d(&tk, c.code[0], EA_HEAD_DIM, Hkv, c.rows, c.outer, cache->kv_str, kDecKeys) ||
        !encode_tmap_u8_4d(&tv, c.code[1], EA_HEAD_DIM, Hkv, c.rows, c.outer, cache->kv_str, kDecKeys))
        return EA_ERR_INVALID_ARG;

    uint8_t *ws = static_cast<uint8_t *>(workspace);
    Q8Args a{};
    a.d.q = static_cast<const __nv_bfloat16 *>(q);
    a.d.q_sb = q_str[0];
    a.d.q_sh = q_str[1];
    a.d.seqlens = seqlens;
    a.d.m = m;
    a.d.unit_first = reinterpret_cast<int32_t *>(ws + L.d.unit_first);
    a.d.unit_splits = reinterpret_cast<int32_t *>(ws + L.d.unit_splits);
    a.d.chunks = reinterpret_cast<int32_t *>(ws + L.d.chunks);
    a.d.part_o = reinterpret_cast<float *>(ws + L.d.partial_o);
    a.d.part_lse = reinterpret_cast<float *>(ws + L.d.partial_lse);
    a.d.hdr = reinterpret_cast<ea_ws_header *>(ws);
    a.d.O = static_cast<__nv_bfloat16 *>(O);
    a.d.o_sb = o_str[0];
    a.d.o_sh = o_str[1];
    a.d.LSE = LSE;
    a.d.B = B;
    a.d.Hq = Hq;
    a.d.Hkv = Hkv;
    a.d.g = Hq / Hkv;
    a.d.Lmax = Lmax;
    a.d.sink = sink < Lmax ? sink : Lmax;
    a.d.window = window < Lmax ? window : Lmax;
    a.d.num_splits = num_splits;
    a.d.max_splits = num_splits > 0 ? num_splits : kQ8MaxSplits;
    a.d.max_chunks = L.max_chunks;
    a.d.whole_waves = 1;
    a.d.num_sms = kQ8Sms;
    a.d.scale_log2 = scale * 1.4426950408889634f;
    a.d.block_mask = block_mask;
    a.d.nBm = static_cast<int>(nBm);
    a.d.blk_count = reinterpret_cast<int32_t *>(ws + L.d.blk_count);
    a.d.blk_list = reinterpret_cast<uint16_t *>(ws + L.d.blk_list);
    a.d.block_table = c.table;
    a.d.bt_stride = c.bt_stride;
    a.d.page_size = c.rows;          // not 0: every tile is 64-key aligned
    a.d.num_pages = c.outer;
    a.d.chunk_min = kQ8MinChunk;
    a.d.chunk_max = kQ8MaxChunk;
    a.ks = c.scale[0];
    a.vs = c.scale[1];
    a.nsb = c.nsb;
    a.log2sb = c.log2sb;
    a.gp = L.gp;
    a.accumulate = accumulate != 0;
    a.key_w = key_weights;
    if (key_weights) {
        a.scores = reinterpret_cast<float *>(ws + L.scores);
        a.lse2 = reinterpret_cast<float *>(ws + L.lse2);
    }

    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return EA_ERR_CUDA;
    const int sms = num_sms(dev);
    if (sms <= 0)
        return EA_ERR_CUDA;
    const int64_t units = static_cast<int64_t>(B) * Hkv;
    const int grid = static_cast<int>(L.max_chunks < sms ? L.max_chunks : sms);
    a.d.self_plan = units <= kSelfPlanUnits ? 1 : 0;
    if (block_mask)
        decode_blocks_kernel<<<static_cast<unsigned>(units), kBlkThreads, 0, st>>>(a.d);
    cudaError_t e = cudaSuccess;
    if (!a.d.self_plan) {
        if (block_mask)
            e = launch_q8_after(decode_plan_kernel, a.d, dim3(1), kPlanThreads, st);
        else
            decode_plan_kernel<<<1, kPlanThreads, 0, st>>>(a.d);
    }
    if (e != cudaSuccess)
        return EA_ERR_CUDA;
    if (c.format == EA_CACHE_E4M3)
        e = key_weights ? launch_q8<true, true>(tk, tv, a, grid, st, dev)
                        : launch_q8<true, false>(tk, tv, a, grid, st, dev);
    else
        e = key_weights ? launch_q8<false, true>(tk, tv, a, grid, st, dev)
                        : launch_q8<false, false>(tk, tv, a, grid, st, dev);
    if (e == cudaSuccess)
        e = launch_q8_merge(a, st);
    if (e == cudaSuccess && key_weights)
        e = launch_q8_after(decode_q8_weights_kernel, a,
                            dim3(static_cast<unsigned>(ceil_div(Lmax, kQ8WKeys)), static_cast<unsigned>(units)),
                            kQ8WThreads, st);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? EA_OK : EA_ERR_CUDA;
}
