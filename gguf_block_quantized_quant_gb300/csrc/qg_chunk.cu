// qg_chunk.cu -- attention of chunks of new tokens over a paged cache on the 5th-generation tensor
// cores: the plan of the row tiles, the kernel, and the merge of items that were cut.
//
// Row r of a sequence is query head g = r % G of a cache head and new token r / G, so the G heads
// that share a cache head share each slot's copy.  A CTA multiplies NQ tiles of 128 rows with tiles
// of BN slots:
//   * producer: one warp copies the key and value tiles through the page table, a tiled TMA copy
//     per page and 128-byte panel (pages end inside a tile); with 8-bit caches four warps fetch
//     the codes instead and write step * code as fp16;
//   * MMA warp: scores S = Q K^T (128 x BN, fp32 in tensor memory), then O += P V with P from
//     tensor memory, where it takes the place of S;
//   * a warpgroup per row tile: each thread owns one row, so its maximum and sum need no
//     exchange; it reads S, writes P = 2^(S - m) and, where the maximum has grown by more than
//     2^8, rescales O.  Up to there a stale maximum is as good: O and the sum carry the same
//     factor and P stays below 2^8.
// With two row tiles (dim 64, 128) one tile's exponentials run under the other's products; with one
// (dim 256, whose O takes half the tensor memory) the scores of the next tile run under them.
// P is rounded to the value's 16-bit type, the operand type of the product: one rounding of
// relative size 2^-12 (2^-9) per factor on average beside that of the result.
//
// Work is counted in slot tiles over all items (row tile, cache head) and cut into one equal range
// per CTA, so causal rows, ragged batches and a few rows over a long context all load the
// machine evenly.  Bound by the tensor cores for long chunks, by the exponentials at dim 64.
#include <algorithm>
#include <mutex>
#include <set>
#include <utility>

#include "qg_attn.cuh"
#include "qg_launch.h"
#include "qg_tcgen05.cuh"
#include "qg_umma.h"

namespace qg {

template <int C, int D>
struct ChunkCfg {
    static constexpr bool Q8 = C == CACHE_Q8;
    static constexpr int NQ = D == 256 ? 1 : 2;  // row tiles
    static constexpr int SB = D == 256 ? 2 : 1;  // score buffers per row tile
    static constexpr int BN = D == 256 ? 64 : 128;
    static constexpr int ROWS = NQ * 128;
    static constexpr int NS = D == 64 ? 6 : 4;   // key/value tiles in shared memory
    static constexpr int NP = D / 64;            // 128-byte panels of a row
    static constexpr uint32_t QB = 128 * D * 2;
    static constexpr uint32_t TILE = BN * D * 2;
    static constexpr int MMA_WARP = 4 * NQ;
    static constexpr int PROD_WARPS = Q8 ? 4 : 1;
    static constexpr int THREADS = (4 * NQ + 1 + PROD_WARPS) * 32;
    static constexpr int NBAR = 2 * NS + NQ + 2 * NQ * SB + NQ;
    static constexpr uint32_t KV_AT = NQ * QB;
    static constexpr uint32_t BAR_AT = KV_AT + NS * TILE;
    static constexpr uint32_t BYTES = BAR_AT + NBAR * 8 + 16 + 1024 /* alignment */;
    // tensor memory columns
    static constexpr int O_COL = NQ * SB * BN;
    static constexpr int COLS = 512;
    static_assert(O_COL + NQ * D <= COLS, "tensor memory");
};

// ----------------------------------------------------------------------------- plan
struct ChunkTile {
    int b, row0, kb0, nt;     // sequence, first row, first slot tile, slot tiles (at least 1)
    int first, n, len, pad;   // Seq of b
};
struct ChunkPlan {
    int64_t *total;    // tiles of all items
    int *nrt;          // row tiles
    int64_t *prefix;   // tiles before each row tile (all cache heads)
    ChunkTile *tile;
};
// Row tiles of a call at most, and the bytes of its plan.
static int64_t chunk_max_tiles(int rows, int G, int tokens, int batch) { return (int64_t)tokens * G / rows + batch; }
static size_t chunk_plan_bytes(int64_t tiles) { return 16 + (size_t)tiles * (sizeof(int64_t) + sizeof(ChunkTile)) + 16; }
static ChunkPlan chunk_plan_at(uint8_t *p, int64_t tiles) {
    ChunkPlan c;
    c.total = reinterpret_cast<int64_t *>(p);
    c.nrt = reinterpret_cast<int *>(p + 8);
    c.tile = reinterpret_cast<ChunkTile *>(p + 16);
    c.prefix = reinterpret_cast<int64_t *>(p + 16 + (size_t)tiles * sizeof(ChunkTile));
    return c;
}

constexpr int PLAN_THREADS = 1024;

// Inclusive prefix of v over the block; sum: the block's total.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *sh, int64_t &sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();
    if (lane == 31) sh[warp] = v;
    __syncthreads();
    int64_t w = lane < PLAN_THREADS / 32 ? sh[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += u;
    }
    sum = __shfl_sync(0xffffffffu, w, 31);
    return v + (warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0);
}

// One block lists the row tiles of all sequences with their slot ranges.
__global__ void __launch_bounds__(PLAN_THREADS) attn_plan_kernel(const AttnArgs a, ChunkPlan p, int rows, int bn, int max_tiles) {
    __shared__ int64_t sh[32];
    __shared__ int off[PLAN_THREADS + 1];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x;
    int64_t cost_before = 0;
    int tiles_before = 0;
    for (int c0 = 0; c0 < a.bt.batch; c0 += PLAN_THREADS) {
        const int nb = min(PLAN_THREADS, a.bt.batch - c0);
        const int mine = tid < nb ? (seq_of(a.bt, c0 + tid).n * a.G + rows - 1) / rows : 0;
        int64_t count;
        const int64_t incl = block_scan(mine, sh, count);
        __syncthreads();
        if (tid == 0) off[0] = 0;
        off[tid + 1] = (int)incl;
        __syncthreads();
        for (int r0 = 0; r0 < (int)count; r0 += PLAN_THREADS) {
            const int r = r0 + tid;
            int64_t cost = 0;
            ChunkTile t{};
            if (r < (int)count) {
                int lo = 0, hi = nb;  // off[lo] <= r < off[hi]
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (off[mid] <= r) lo = mid; else hi = mid;
                }
                const Seq s = seq_of(a.bt, c0 + lo);
                t.b = c0 + lo;
                t.row0 = (r - off[lo]) * rows;
                t.first = s.first, t.n = s.n, t.len = s.len;
                const int tf = t.row0 / a.G, tl = (min(t.row0 + rows, s.n * a.G) - 1) / a.G;  // first, last token
                const int from = a.window ? max(0, s.len - s.n + tf - a.window + 1) : 0;
                const int end = s.len - s.n + tl + 1;  // slots that the last row sees
                t.kb0 = from / bn;
                t.nt = max(1, (end + bn - 1) / bn - t.kb0);
                // q_start that decreases could list more tiles than the call's tokens make: those are left out
                if (tiles_before + r < max_tiles) cost = (int64_t)t.nt * a.Hk;
            }
            int64_t sum;
            const int64_t inc = block_scan(cost, sh, sum);
            const int at = tiles_before + r;
            if (r < (int)count && at < max_tiles) {
                p.tile[at] = t;
                p.prefix[at] = cost_before + inc - cost;
            }
            cost_before += sum;
        }
        tiles_before += (int)count;
        __syncthreads();
    }
    if (tid == 0) {
        *p.total = cost_before;
        *p.nrt = min(tiles_before, max_tiles);
    }
}

// Position in the work list: every role of a CTA walks it by itself.
struct ChunkWalk {
    ChunkTile t;
    int rt, h, blk;
    int64_t left;  // tiles left in this CTA's range
};
__device__ __forceinline__ ChunkTile chunk_tile(const ChunkPlan &p, int rt) {
    const int4 x = reinterpret_cast<const int4 *>(p.tile + rt)[0], y = reinterpret_cast<const int4 *>(p.tile + rt)[1];
    return ChunkTile{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
}
// The position of tile `at` of the list; whole warp.
__device__ __forceinline__ ChunkWalk chunk_find(const ChunkPlan &p, int nrt, int64_t at) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = nrt;  // the row tile is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const unsigned m = __ballot_sync(0xffffffffu, lane * step < n && (lane == 0 || p.prefix[lo + lane * step] <= at));
        const int last = __popc(m) - 1;
        lo += last * step;
        n = min(step, n - last * step);
    }
    ChunkWalk k;
    k.t = chunk_tile(p, lo);
    const int64_t rem = at - p.prefix[lo];
    k.rt = lo;
    k.h = (int)(rem / k.t.nt);
    k.blk = (int)(rem % k.t.nt);
    k.left = 0;
    return k;
}
__device__ __forceinline__ int chunk_end(const ChunkWalk &k) { return (int)min((int64_t)k.t.nt, k.blk + k.left); }
__device__ __forceinline__ void chunk_next(ChunkWalk &k, const ChunkPlan &p, int Hk, int taken) {
    k.left -= taken;
    k.blk += taken;
    if (k.left <= 0 || k.blk < k.t.nt) return;
    k.blk = 0;
    if (++k.h < Hk) return;
    k.h = 0;
    k.t = chunk_tile(p, ++k.rt);
}
__device__ __forceinline__ int chunk_ctas(int64_t total, int max_ctas) {
    return (int)min((int64_t)max_ctas, max((int64_t)1, total));
}
// CTA c takes the tiles from start(c).
__device__ __forceinline__ int64_t chunk_start(int64_t total, int ctas, int c) {
    return total / ctas * c + (int)(total % ctas) * c / ctas;
}

// ----------------------------------------------------------------------------- kernel
template <int C, int D>
__global__ void __launch_bounds__(ChunkCfg<C, D>::THREADS, 1)
    attn_chunk_kernel(const AttnArgs a, const ChunkPlan plan, int box_rows, uint32_t qsign, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap) {
    using Cfg = ChunkCfg<C, D>;
    using T = typename CacheT<C>::Q;
    constexpr int NQ = Cfg::NQ, SB = Cfg::SB, BN = Cfg::BN, NS = Cfg::NS;
    constexpr bool BF = C == CACHE_BF16;
    extern __shared__ __align__(16) uint8_t ck_smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (smem_addr(ck_smem) + 1023u) & ~1023u;
    const uint32_t kv0 = base + Cfg::KV_AT, bars = base + Cfg::BAR_AT;
    auto kv_full = [&](int s) { return bars + 8u * s; };
    auto kv_empty = [&](int s) { return bars + 8u * (NS + s); };
    auto q_full = [&](int q) { return bars + 8u * (2 * NS + q); };
    auto s_full = [&](int q, int b) { return bars + 8u * (2 * NS + NQ + q * SB + b); };
    auto p_full = [&](int q, int b) { return bars + 8u * (2 * NS + NQ + NQ * SB + q * SB + b); };
    auto pv_done = [&](int q) { return bars + 8u * (2 * NS + NQ + 2 * NQ * SB + q); };
    const uint32_t taddr_slot = bars + 8u * Cfg::NBAR;

    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(kv_full(s), Cfg::Q8 ? 128 : 1);
            mbar_init(kv_empty(s), 1);
        }
        for (int q = 0; q < NQ; ++q) {
            mbar_init(q_full(q), 128);
            mbar_init(pv_done(q), 1);
            for (int b = 0; b < SB; ++b) {
                mbar_init(s_full(q, b), 1);
                mbar_init(p_full(q, b), 128);
            }
        }
        fence_mbar_init();
    }
    if (warp == Cfg::MMA_WARP) tmem_alloc(taddr_slot, Cfg::COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = lds32(taddr_slot);
    griddep_wait();
    griddep_launch_dependents();

    const int64_t total = *plan.total;
    const int ctas = chunk_ctas(total, gridDim.x);
    const int64_t w0 = (int)blockIdx.x < ctas ? chunk_start(total, ctas, blockIdx.x) : 0;
    const int64_t w1 = (int)blockIdx.x < ctas ? chunk_start(total, ctas, blockIdx.x + 1) : 0;
    ChunkWalk k;
    k.left = 0;
    if (w1 > w0) {
        k = chunk_find(plan, *plan.nrt, w0);
        k.left = w1 - w0;
    }
    uint32_t units = 0;  // key and value tiles so far: tile u sits in slot u % NS

    if (warp < 4 * NQ) {
        // ------------------------------------------------------------ a row per thread
        const int q = warp >> 2, r = tid & 127;
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t ocol = lanes + Cfg::O_COL + q * D;
        uint32_t done = 0;  // slot tiles of this row tile so far
        while (k.left > 0) {
            const int end = chunk_end(k), taken = end - k.blk;
            const int nrows = k.t.n * a.G, row0 = k.t.row0 + 128 * q;
            if (row0 < nrows) {
                // ---- the queries into shared memory (the products that read the last ones are complete)
                constexpr int CPR = D / 8;  // 16-byte chunks of a row
#pragma unroll 8
                for (int i = 0; i < CPR; ++i) {
                    const int x = i * 128 + r, row = x / CPR, ch = x % CPR, rr = row0 + row;
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (rr < nrows) {
                        v = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.q) + (int64_t)(k.t.first + rr / a.G) * a.ldq +
                                                             (int64_t)(k.h * a.G + rr % a.G) * a.hdq + 8 * ch);
                        v.x ^= qsign, v.y ^= qsign, v.z ^= qsign, v.w ^= qsign;
                    }
                    sts128(base + q * Cfg::QB + (ch >> 3) * (128 * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4), v.x, v.y, v.z, v.w);
                }
                fence_proxy_async_smem();
                mbar_arrive(q_full(q));

                const int rr = row0 + r, pos0 = k.t.len - k.t.n;
                const int pos = pos0 + rr / a.G;
                const int hi = rr < nrows ? pos : -1, lo = a.window ? max(0, pos - a.window + 1) : 0;
                const int hi_min = pos0 + row0 / a.G;  // every row sees up to here, and from lo_max on
                const int lo_max = a.window ? max(0, pos0 + (min(row0 + 128, nrows) - 1) / a.G - a.window + 1) : 0;
                float m = -INFINITY, l = 0.0f;
                for (int j = k.blk; j < end; ++j, ++done) {
                    const int buf = SB == 1 ? 0 : (int)(done & 1);
                    const uint32_t scol = lanes + (q * SB + buf) * BN;
                    const int key0 = (k.t.kb0 + j) * BN;
                    const int c_hi = hi - key0, c_lo = lo - key0;  // visible columns
                    const bool edge = key0 + BN - 1 > hi_min || key0 < lo_max;
                    mbar_wait(s_full(q, buf), (done / SB) & 1);
                    tc_fence_after();
                    uint32_t s[2][32];
                    float mx = -INFINITY;
                    auto mask = [&](uint32_t (&v)[32], int c0) {
                        if (edge) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (c0 + i > c_hi || c0 + i < c_lo) v[i] = 0xff800000u;  // -inf
                        }
                    };
                    tmem_ld32(scol, s[0]);
#pragma unroll
                    for (int c = 0; c < BN / 32; ++c) {
                        tmem_wait_ld(s[c & 1]);
                        if (c + 1 < BN / 32) tmem_ld32(scol + 32 * (c + 1), s[(c + 1) & 1]);
                        mask(s[c & 1], 32 * c);
                        float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i & 3] = fmaxf(x[i & 3], __uint_as_float(s[c & 1][i]));
                        mx = fmaxf(mx, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
                    }
                    // ---- rescale where some row of the warp needs it (the first tile starts O afresh)
                    if (j == k.blk) {
                        m = mx;
                    } else {
                        const bool grown = (mx - m) * a.scale2 > 8.0f || (m == -INFINITY && mx > m);
                        if (__any_sync(0xffffffffu, grown)) {
                            const float mn = fmaxf(m, mx), f = mn > m ? exp2_approx((m - mn) * a.scale2) : 1.0f;
                            m = mn;
                            l *= f;
                            mbar_wait(pv_done(q), (done - 1) & 1);
                            tc_fence_after();
#pragma unroll
                            for (int c = 0; c < D; c += 32) {
                                uint32_t o[32];
                                tmem_ld32(ocol + c, o);
                                tmem_wait_ld(o);
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                tmem_st32(ocol + c, o);
                            }
                            tmem_wait_st();
                        }
                    }
                    const float mz = (m == -INFINITY ? 0.0f : m) * a.scale2;
                    // ---- P over S: chunk c of 32 scores becomes columns 16 c .. 16 c + 15, which were read before
                    float sum[4] = {};
                    tmem_ld32(scol, s[0]);
#pragma unroll
                    for (int c = 0; c < BN / 32; ++c) {
                        tmem_wait_ld(s[c & 1]);
                        if (c + 1 < BN / 32) tmem_ld32(scol + 32 * (c + 1), s[(c + 1) & 1]);
                        mask(s[c & 1], 32 * c);
                        uint32_t p[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float p0 = exp2_approx(fmaf(__uint_as_float(s[c & 1][2 * i]), a.scale2, -mz));
                            const float p1 = exp2_approx(fmaf(__uint_as_float(s[c & 1][2 * i + 1]), a.scale2, -mz));
                            sum[(2 * i) & 3] += p0;
                            sum[(2 * i + 1) & 3] += p1;
                            p[i] = pack2<T>(p0, p1);
                        }
                        tmem_st16(scol + 16 * c, p);
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(p_full(q, buf));
                }
                // ---- result.  A full score buffer says that the products SB tiles back are complete, so
                // the wait for the last ones must not take an older phase of the same parity for them
                if (SB == 2 && taken > 1) mbar_wait(pv_done(q), done & 1);
                mbar_wait(pv_done(q), (done - 1) & 1);
                tc_fence_after();
                const bool whole = k.blk == 0 && end == k.t.nt;
                const float inv = l > 0.0f ? 1.0f / l : l;  // nothing visible: 0
                const float ls = l > 0.0f ? (m == -INFINITY ? 0.0f : m) * a.scale2 + log2_approx(l) : l == 0.0f ? -INFINITY : l;
                float *part = a.part + (size_t)(2 * blockIdx.x + (k.blk == 0 ? 1 : 0)) * attn_part_floats(Cfg::ROWS, D);
                const int pr = 128 * q + r;
                const int64_t orow = (int64_t)(k.t.first + rr / a.G) * a.Hq + k.h * a.G + rr % a.G;
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(ocol + c, o);
                    tmem_wait_ld(o);
                    if (rr < nrows) {
                        float v[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(o[i]) * inv;
                        if (!whole)
                            store_vec<float, 32>(part + (size_t)pr * D + c, v);
                        else if (a.out_f32)
                            store_vec<float, 32>(static_cast<float *>(a.out) + orow * D + c, v);
                        else
                            store_vec<T, 32>(static_cast<T *>(a.out) + orow * D + c, v);
                    }
                }
                if (rr < nrows) {
                    if (!whole)
                        part[(size_t)Cfg::ROWS * D + pr] = ls;
                    else if (a.lse)
                        a.lse[orow] = ls * LN2;
                }
                tc_fence_before();  // the next item's products overwrite O once its P arrives
            }
            chunk_next(k, plan, a.Hk, taken);
        }
    } else if (warp == Cfg::MMA_WARP) {
        // ------------------------------------------------------------ products
        constexpr uint32_t id_s = umma_idesc_16(128, BN, BF, false), id_o = umma_idesc_16(128, D, BF, true);
        uint32_t items[NQ] = {}, done[NQ] = {};
        while (k.left > 0) {
            const int end = chunk_end(k), taken = end - k.blk;
            const int nrows = k.t.n * a.G;
            const int live = NQ == 1 || k.t.row0 + 128 >= nrows ? 1 : NQ;
            const uint32_t u0 = units;
            const int seen_lo = a.window ? max(0, k.t.len - k.t.n + k.t.row0 / a.G - a.window + 1) : 0;
#pragma unroll
            for (int q = 0; q < NQ; ++q)
                if (q < live) {
                    mbar_wait(q_full(q), items[q] & 1);
                    ++items[q];
                }
            tc_fence_after();
            auto scores = [&](int q, int j) {  // S = Q K^T of slot tile j of the segment
                const uint32_t u = u0 + 2 * j, slot = u % NS, n = done[q] + j;
                if (q == 0) {
                    mbar_wait(kv_full(slot), (u / NS) & 1);
                    tc_fence_after();
                }
                if (lane == 0) {
                    const uint64_t qd = umma_desc_kmajor_sw128(base + q * Cfg::QB), kd = umma_desc_kmajor_sw128(kv0 + slot * Cfg::TILE);
                    const uint32_t buf = SB == 1 ? 0 : (n & 1);
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
                        umma_f16(tmem + (q * SB + buf) * BN, qd + (uint64_t)((i / 4) * (128 * 128 / 16) + 2 * (i % 4)),
                                 kd + (uint64_t)((i / 4) * (BN * 128 / 16) + 2 * (i % 4)), id_s, i != 0);
                    umma_commit(s_full(q, buf));
                    if (q == live - 1) umma_commit(kv_empty(slot));
                }
                __syncwarp();
            };
            auto product = [&](int q, int j) {  // O += P V
                const uint32_t u = u0 + 2 * j + 1, slot = u % NS, n = done[q] + j;
                const uint32_t buf = SB == 1 ? 0 : (n & 1), vt = kv0 + slot * Cfg::TILE;
                if (q == 0) {
                    mbar_wait(kv_full(slot), (u / NS) & 1);
                    if (!Cfg::Q8) {
                        // slots that no row sees may hold anything: their values are taken as zero
                        const int key0 = (k.t.kb0 + k.blk + j) * BN;
                        const int z0 = min(BN, max(0, seen_lo - key0)), z1 = min(BN, max(0, k.t.len - key0));
                        if (z0 > 0 || z1 < BN) {
                            for (int x = lane; x < (z0 + BN - z1) * (D / 8); x += 32) {
                                const int row = x / (D / 8), ch = x % (D / 8);
                                sts128(vt + (ch >> 3) * (BN * 128) + (row < z0 ? row : row - z0 + z1) * 128 + (ch & 7) * 16, 0u, 0u, 0u, 0u);
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                    }
                }
                mbar_wait(p_full(q, buf), (n / SB) & 1);
                tc_fence_after();
                if (lane == 0) {
                    const uint64_t vd = umma_desc_mnmajor_sw128(vt, BN * 128);
#pragma unroll
                    for (int i = 0; i < BN / 16; ++i)
                        umma_f16_ta(tmem + Cfg::O_COL + q * D, tmem + (q * SB + buf) * BN + 8 * i, vd + (uint64_t)(i * (2048 / 16)), id_o,
                                    j != 0 || i != 0);
                    umma_commit(pv_done(q));
                    if (q == live - 1) umma_commit(kv_empty(slot));
                }
                __syncwarp();
            };
            if constexpr (SB == 1) {
                for (int q = 0; q < live; ++q) scores(q, 0);
                for (int j = 0; j < taken; ++j)
                    for (int q = 0; q < live; ++q) {
                        product(q, j);
                        if (j + 1 < taken) scores(q, j + 1);
                    }
            } else {
                scores(0, 0);
                for (int j = 0; j < taken; ++j) {
                    if (j + 1 < taken) scores(0, j + 1);
                    product(0, j);
                }
            }
#pragma unroll
            for (int q = 0; q < NQ; ++q)
                if (q < live) done[q] += taken;
            units += 2 * taken;
            chunk_next(k, plan, a.Hk, taken);
        }
        if (lane == 0) {
            // complete already on the normal path; after a wait gave up, let products in flight end
#pragma unroll
            for (int q = 0; q < NQ; ++q)
                if (done[q]) mbar_drain(pv_done(q), (done[q] - 1) & 1, DRAIN_NS);
        }
        __syncwarp();
    } else if constexpr (!Cfg::Q8) {
        // ------------------------------------------------------------ copies: lane = (box of slots, panel)
        const int boxes = BN / box_rows, box = lane / Cfg::NP, panel = lane % Cfg::NP;
        const bool on = box < boxes;
        while (k.left > 0) {
            const int end = chunk_end(k), taken = end - k.blk;
            for (int j = k.blk; j < end; ++j) {
                const int key = (k.t.kb0 + j) * BN + box * box_rows;
                int page = a.bt.n_pages;  // out of range: zeros
                if (on && key < k.t.len) {
                    page = a.bt.pages[k.t.b * a.bt.table_stride + key / a.bt.page];
                    if ((unsigned)page >= (unsigned)a.bt.n_pages) page = a.bt.n_pages;
                }
#pragma unroll
                for (int v = 0; v < 2; ++v, ++units) {
                    const uint32_t slot = units % NS;
                    if (units >= NS) mbar_wait(kv_empty(slot), (units / NS - 1) & 1);
                    if (lane == 0) mbar_arrive_expect_tx(kv_full(slot), Cfg::TILE);
                    __syncwarp();
                    if (on)
                        tma_load_4d(kv0 + slot * Cfg::TILE + panel * (BN * 128) + box * box_rows * 128, v ? &vmap : &kmap, 64 * panel,
                                    key % a.bt.page, k.h, page, kv_full(slot));
                }
            }
            chunk_next(k, plan, a.Hk, taken);
        }
        if (lane == 0)
            for (uint32_t s = 0; s < NS && s < units; ++s)
                mbar_drain(kv_full(s), ((units - 1 - s) / NS) & 1, DRAIN_NS);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ 8-bit codes to fp16 tiles
        const int ct = tid - (Cfg::MMA_WARP + 1) * 32;
        constexpr int PER = BN * D / 16 / 128;  // 16-code chunks per thread
        constexpr int CPR = D / 16;
        struct Raw {
            uint4 c[PER];
            uint16_t d[PER];
        };
        Raw kr, vr;
        ChunkWalk nx = k;  // the tile to fetch next
        int nj = k.blk;
        auto fetch = [&](Raw &w, bool val) {  // codes and steps of the key (value) tile at (nx, nj)
            if (nx.left <= 0) return;
            const int seen_lo = a.window ? max(0, nx.t.len - nx.t.n + nx.t.row0 / a.G - a.window + 1) : 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int x = i * 128 + ct, row = x / CPR, ch = x % CPR, key = (nx.t.kb0 + nj) * BN + row;
                w.c[i] = make_uint4(0u, 0u, 0u, 0u);
                w.d[i] = 0;
                if (key >= seen_lo && key < nx.t.len) {
                    const int page = a.bt.pages[nx.t.b * a.bt.table_stride + key / a.bt.page], slot = key % a.bt.page;
                    if ((unsigned)page < (unsigned)a.bt.n_pages) {
                        w.c[i] = *reinterpret_cast<const uint4 *>(static_cast<const int8_t *>(val ? a.vc : a.kc) + page * a.page_stride +
                                                                  nx.h * a.head_stride + slot * a.slot_stride + 16 * ch);
                        w.d[i] = reinterpret_cast<const uint16_t *>(val ? a.vd : a.kd)[page * a.step_stride +
                                                                                      ((int64_t)nx.h * a.bt.page + slot) * (D / 32) + ch / 2];
                    }
                }
            }
        };
        auto put = [&](const Raw &w) {
            const uint32_t slot = units % NS;
            if (units >= NS) mbar_wait(kv_empty(slot), (units / NS - 1) & 1);
            ++units;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int x = i * 128 + ct, row = x / CPR, ch = x % CPR;
                const uint32_t dd = w.d[i] | (uint32_t)w.d[i] << 16;
                const uint32_t in[4] = {w.c[i].x, w.c[i].y, w.c[i].z, w.c[i].w};
                uint32_t h[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t b = in[e] ^ 0x80808080u;
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t c = codes_to_f16(b, y ? 0x4342 : 0x4140);
                        const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&c), *reinterpret_cast<const __half2 *>(&dd));
                        h[2 * e + y] = *reinterpret_cast<const uint32_t *>(&r);
                    }
                }
                const uint32_t row_at = kv0 + slot * Cfg::TILE + (ch >> 2) * (BN * 128) + row * 128;
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    sts128(row_at + (((2 * (ch & 3) + y) ^ (row & 7)) << 4), h[4 * y], h[4 * y + 1], h[4 * y + 2], h[4 * y + 3]);
            }
            fence_proxy_async_smem();
            mbar_arrive(kv_full(slot));
        };
        fetch(kr, false);
        fetch(vr, true);
        while (k.left > 0) {
            const int end = chunk_end(k), taken = end - k.blk;
            for (int j = k.blk; j < end; ++j) {
                if (++nj >= chunk_end(nx)) {
                    chunk_next(nx, plan, a.Hk, nj - nx.blk);
                    nj = nx.blk;
                }
                put(kr);
                fetch(kr, false);
                put(vr);
                fetch(vr, true);
            }
            chunk_next(k, plan, a.Hk, taken);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == Cfg::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, Cfg::COLS);
    }
}

// Merges the partial results of the items that range boundaries cut: as attn_join_kernel, block
// (x, y) for the item cut by boundary x + 1 and rows 8 y .. 8 y + 7, one per warp.
template <class T, int D>
__global__ void __launch_bounds__(256) attn_chunk_join_kernel(const AttnArgs a, const ChunkPlan plan, int max_ctas) {
    constexpr int ROWS = ChunkCfg<CACHE_F16, D>::ROWS, V = D / 32;
    griddep_wait();
    griddep_launch_dependents();
    const int64_t total = *plan.total;
    const int ctas = chunk_ctas(total, max_ctas), bound = (int)blockIdx.x + 1;
    if (bound >= ctas) return;
    const int64_t at = chunk_start(total, ctas, bound);
    const ChunkWalk k = chunk_find(plan, *plan.nrt, at);
    if (k.blk == 0) return;
    const int64_t s0 = at - k.blk, s1 = s0 + k.t.nt;
    if (bound > 1 && chunk_start(total, ctas, bound - 1) > s0) return;  // an earlier boundary joins it
    const int lane = threadIdx.x & 31, r = blockIdx.y * 8 + (threadIdx.x >> 5), rr = k.t.row0 + r;
    if (rr >= k.t.n * a.G) return;
    auto part = [&](int c) {
        return a.part + (size_t)(2 * c + (c == bound - 1 ? 1 : 0)) * attn_part_floats(ROWS, D);
    };
    int last = bound;
    while (last + 1 < ctas && chunk_start(total, ctas, last + 1) < s1) ++last;
    float mx = -INFINITY;
    for (int c = bound - 1; c <= last; ++c) mx = fmaxf(mx, part(c)[(size_t)ROWS * D + r]);
    const float mz = mx == -INFINITY ? 0.0f : mx;
    float sum = 0.0f, v[V] = {};
#pragma unroll 2
    for (int c = bound - 1; c <= last; ++c) {
        const float *p = part(c);
        const float w = exp2_approx(p[(size_t)ROWS * D + r] - mz);
        float x[V];
        load_vec<float, V>(p + (size_t)r * D + lane * V, x);
        sum += w;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = fmaf(w, x[i], v[i]);
    }
    const float inv = sum > 0.0f ? 1.0f / sum : sum;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] *= inv;
    const int64_t row = (int64_t)(k.t.first + rr / a.G) * a.Hq + k.h * a.G + rr % a.G;
    if (a.out_f32)
        store_vec<float, V>(static_cast<float *>(a.out) + row * D + lane * V, v);
    else
        store_vec<T, V>(static_cast<T *>(a.out) + row * D + lane * V, v);
    if (a.lse && lane == 0) a.lse[row] = sum > 0.0f ? (mz + log2_approx(sum)) * LN2 : sum == 0.0f ? -INFINITY : sum;
}

// ----------------------------------------------------------------------------- host
static int chunk_rows(int D) { return D == 256 ? 128 : 256; }

size_t attn_chunk_workspace(int D, int G, int tokens, int batch, int sms) {
    const int rows = chunk_rows(D);
    const size_t parts = (size_t)sms * 2 * attn_part_floats(rows, D) * sizeof(float);
    return parts + chunk_plan_bytes(chunk_max_tiles(rows, G, tokens, batch));
}

static int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

template <int C, int D>
static int chunk_run(const AttnArgs &in, const qg_paged &c, uint8_t *ws, int sms, cudaStream_t s) {
    using Cfg = ChunkCfg<C, D>;
    using T = typename CacheT<C>::Q;
    static_assert(Cfg::BYTES <= SMEM_MAX, "shared memory of the chunk kernel");
    AttnArgs a = in;
    a.part = reinterpret_cast<float *>(ws);
    const int64_t tiles = chunk_max_tiles(Cfg::ROWS, a.G, a.bt.tokens, a.bt.batch);
    const ChunkPlan plan = chunk_plan_at(ws + (size_t)sms * 2 * attn_part_floats(Cfg::ROWS, D) * sizeof(float), tiles);
    // the maximum is taken over unscaled scores: a negative scale goes into the queries' signs, and
    // a scale of zero is a small one (masked scores stay -inf)
    const uint32_t qsign = a.scale2 < 0.0f ? 0x80008000u : 0u;
    a.scale2 = std::max(std::abs(a.scale2), 1e-30f);
    const int box = gcd(c.page, Cfg::BN);
    CUtensorMap km{}, vm{};
    if (!Cfg::Q8 && (!attn_tensor_map(&km, c, c.k, box) || !attn_tensor_map(&vm, c, c.v, box))) return QG_ECUDA;
    if (!launch_programmatic(attn_plan_kernel, dim3(1), PLAN_THREADS, 0, s, a, plan, Cfg::ROWS, Cfg::BN, (int)tiles)) return QG_ECUDA;
    auto kern = attn_chunk_kernel<C, D>;
    if (!allow_smem((const void *)kern, Cfg::BYTES)) return QG_ECUDA;
    if (!launch_programmatic(kern, dim3((unsigned)sms), Cfg::THREADS, Cfg::BYTES, s, a, plan, box, qsign, km, vm)) return QG_ECUDA;
    if (sms == 1) return QG_OK;
    auto join = attn_chunk_join_kernel<T, D>;
    return launch_programmatic(join, dim3((unsigned)(sms - 1), Cfg::ROWS / 8), 256, 0, s, a, plan, sms) ? QG_OK : QG_ECUDA;
}

template <int C>
static int chunk_dim(const AttnArgs &a, const qg_paged &c, uint8_t *ws, int sms, cudaStream_t s) {
    return c.dim == 64 ? chunk_run<C, 64>(a, c, ws, sms, s) : c.dim == 128 ? chunk_run<C, 128>(a, c, ws, sms, s) : chunk_run<C, 256>(a, c, ws, sms, s);
}
int attn_chunk(const AttnArgs &a, const qg_paged &c, uint8_t *ws, int sms, cudaStream_t s) {
    return c.type == QG_F16    ? chunk_dim<CACHE_F16>(a, c, ws, sms, s)
           : c.type == QG_BF16 ? chunk_dim<CACHE_BF16>(a, c, ws, sms, s)
                               : chunk_dim<CACHE_Q8>(a, c, ws, sms, s);
}

int attn_chunk_dev_err_take(unsigned int *err) {
    unsigned int zero = 0;
    if (cudaMemcpyFromSymbol(err, g_qg_dev_err, sizeof(*err)) != cudaSuccess) return QG_ECUDA;
    if (cudaMemcpyToSymbol(g_qg_dev_err, &zero, sizeof(zero)) != cudaSuccess) return QG_ECUDA;
    return QG_OK;
}

}  // namespace qg
