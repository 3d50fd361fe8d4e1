// qg_attn.cu -- attention over a paged cache: the C entry points, the kernel for few rows per
// sequence (single tokens, short chunks) and the kernel that joins partial results.
#include <algorithm>
#include <mutex>
#include <set>
#include <utility>

#include "qg_attn.cuh"
#include "qg_launch.h"

namespace qg {

// ----------------------------------------------------------------------------- few rows
// Row r of a tile is query head g = r % G of the tile's cache head and new token r / G, so the
// G heads that share a cache head read its slots once.  Work is counted in blocks of 16 slots
// over all (sequence, cache head, row tile) items and cut into one equal range per CTA: a long
// sequence spreads over many CTAs and many short ones share a CTA.  An item cut by a range
// boundary leaves partial results, which the join kernel merges in a fixed order.
//
// Inside a range each warp takes every NW-th block.  It has its own ring of slots in shared
// memory, filled by tiled TMA copies that it issues itself S blocks ahead (also across items),
// and its own running maximum and sum, so warps meet only at the end of an item.
//
// Scores and value sums are m16n8k16 products with the cache as the 16-row operand: S^T = K Q^T
// (16 slots x 8 rows) and O^T += V^T P^T (16 columns x 8 rows).  Eight query rows then fill a
// product; with the rows as the 16-row operand half of each would be padding for the usual 4 to 8
// heads per cache head, at twice the accumulators.  NR = 2 takes 16 rows.  P^T changes from
// accumulator to operand layout by a transposing move within the warp.
//
// Bound by the read of the cache; the products take a small part of that time, which is why the
// probabilities can go in as two addends (hi + lo): over a 16-bit cache the value sums are then those of
// factors of 22 (16) bits instead of the 11 (8) of one fp16 (bf16) factor.  8-bit keys are whole numbers in the
// products, their steps applied to the sums of 32 in fp32; 8-bit values go in as step * code rounded once
// to fp16 (relative 2^-12 on average, 2^-11 at most), as their step, one per 32 columns of a slot, has no place
// in a factor that all columns share.
//
// 64 ragged sequences of 300 to 16000 slots, 32/8 heads of 128, bf16: 156 us, 0.93 of the measured copy
// bandwidth; 4 new tokens each in fp16 (16 rows) 231 us (0.82).  8-bit caches are bound by the latency of each
// warp's chain from codes to fp16 pairs to products, with three or four warps a scheduler and half of the
// issue slots in use: 48 sequences of 100 to 12000, 24/4 heads of 256, 60 us (0.59); one of 32000 19.7 us.
// One of 700 9.3 us, as long in a graph: two launches that wait for each other and a chain of loads.
constexpr int DEC_ROWS = 16;     // rows of a tile at most (NR = 2)
constexpr int DEC_BLK = 16;      // slots per block: the least page size
// An item costs its blocks and a fixed part more, in the same unit, for its queries, its last incomplete
// round of the warps and their merge; a range that ends inside that part leaves the item to the
// next CTA.  Measured on 64 (48) ragged sequences of 300 to 16000 (100 to 12000) slots, fp16 with dim
// 128 (8-bit with dim 256), us: 162 (83) with 6 (12), 159 (65.5) with 12 (24), 158 (63) with 20 (36).
constexpr int dec_ov(bool q8) { return q8 ? 32 : 16; }
constexpr int DEC_MIN_BLKS = 8;  // blocks a CTA takes at least

template <int C, int D, int NR>
struct DecCfg {
    static constexpr bool Q8 = C == CACHE_Q8;
    static constexpr int ROWS = 8 * NR;
    static constexpr int ES = Q8 ? 1 : 2;
    static constexpr int ROWB = D * ES;                      // bytes of a slot's row
    static constexpr int PANEL = ROWB < 128 ? ROWB : 128;    // bytes of a swizzled panel row
    static constexpr int NP = ROWB / PANEL;                  // panels
    static constexpr int TILE = DEC_BLK * ROWB;              // K (or V) bytes of a block
    static constexpr int STEPS = Q8 ? DEC_BLK * (D / 32) * 2 : 0;
    // Warps and ring slots: about 190 KB in flight per SM; 8-bit codes take more instructions per byte
    // and get more warps where the accumulators leave registers for them
    static constexpr int NW = D == 256 ? (Q8 ? (NR == 1 ? 12 : 8) : 6) : D == 128 ? (Q8 ? (NR == 1 ? 16 : 12) : 8) : (Q8 ? 16 : 12);
    static constexpr int MW = D == 256 && Q8 ? 32 : 64;      // columns merged at a time
    static constexpr int ROOM = (222 * 1024 - NW * ROWS * (MW * 4 + 8) - (Q8 ? NR * D * 16 : 0)) / (NW * 2 * (TILE + STEPS));
    static constexpr int S = ROOM > 8 ? 8 : ROOM;
    static constexpr uint32_t RING = (uint32_t)NW * S * 2 * TILE;
    static constexpr uint32_t STEP_AT = RING;
    static constexpr uint32_t MERGE_AT = STEP_AT + (uint32_t)NW * S * 2 * STEPS;
    static constexpr uint32_t ML_AT = MERGE_AT + (uint32_t)NW * ROWS * MW * 4;
    static constexpr uint32_t QS_AT = ML_AT + (uint32_t)NW * ROWS * 8;  // 8-bit: the item's queries, 16 bytes per lane and 32-element block
    static constexpr uint32_t QS = Q8 ? NR * (D / 32) * 512 : 0;
    static constexpr uint32_t BAR_AT = QS_AT + QS;
    static constexpr uint32_t BYTES = BAR_AT + (uint32_t)NW * S * 8 + 1024 /* alignment */;
    static_assert(MERGE_AT % 16 == 0 && ML_AT % 8 == 0 && QS_AT % 16 == 0 && BAR_AT % 8 == 0 && S >= 2, "layout");
};

// The blocks of one sequence: every item (cache head, row tile) of it has the same slots.
template <int ROWS, int OV>
struct SeqWork {
    Seq sq;
    int nrt;        // row tiles
    int kb0, nblk;  // first block of 16 slots and their number (at least 1)
    __device__ __forceinline__ SeqWork() {}
    __device__ __forceinline__ SeqWork(const AttnArgs &a, int b) : sq(seq_of(a.bt, b)) {
        nrt = (sq.n * a.G + ROWS - 1) / ROWS;
        const int low = seen_from(sq.len - sq.n, a.window);
        kb0 = low / DEC_BLK;
        nblk = max(1, (sq.len + DEC_BLK - 1) / DEC_BLK - kb0);
    }
    __device__ __forceinline__ int64_t cost(const AttnArgs &a) const { return (int64_t)nrt * a.Hk * (nblk + OV); }
};

// Position in the work list.
template <int ROWS, int OV>
struct Walk {
    SeqWork<ROWS, OV> w;
    int b, item, u;  // item: cache head * nrt + row tile; unit of the item
    int64_t left;    // units left in this CTA's range
    __device__ __forceinline__ int blk() const { return max(0, u - OV); }  // first block of the segment
    __device__ __forceinline__ int end() const { return (int)min((int64_t)w.nblk, max((int64_t)0, u + left - OV)); }
    __device__ __forceinline__ void next(const AttnArgs &a) {  // on to the next item; left is 0 at the range's end
        left -= w.nblk + OV - u;
        u = 0;
        if (left <= OV) {  // a rest of OV units or less holds no block
            left = 0;
            return;
        }
        if (++item < w.nrt * a.Hk) return;
        item = 0;
        do {
            w = SeqWork<ROWS, OV>(a, ++b);
        } while (w.nrt == 0);  // left > 0: a later sequence has work
    }
};

// Units of all sequences, and the CTAs that share them.  Whole warp: lane i takes every 32nd sequence.
template <int ROWS, int OV>
__device__ __forceinline__ int64_t walk_total(const AttnArgs &a, int &ctas) {
    int64_t units = 0, items = 0;
    for (int b = threadIdx.x & 31; b < a.bt.batch; b += 32) {
        const SeqWork<ROWS, OV> w(a, b);
        units += w.cost(a);
        items += (int64_t)w.nrt * a.Hk;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        units += __shfl_xor_sync(0xffffffffu, units, o);
        items += __shfl_xor_sync(0xffffffffu, items, o);
    }
    ctas = (int)min((int64_t)gridDim.x, max((int64_t)1, (units - items * OV) / DEC_MIN_BLKS));
    return units;
}
// The position of unit `at` (below the total); whole warp.
template <int ROWS, int OV>
__device__ __forceinline__ Walk<ROWS, OV> walk_find(const AttnArgs &a, int64_t at) {
    const int lane = threadIdx.x & 31;
    Walk<ROWS, OV> k;
    int64_t base = 0, rem = 0;
    for (int c0 = 0;; c0 += 32) {  // ends: at is below the total
        const int64_t cost = c0 + lane < a.bt.batch ? SeqWork<ROWS, OV>(a, c0 + lane).cost(a) : 0;
        int64_t v = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        const unsigned m = __ballot_sync(0xffffffffu, base + v > at);
        if (m || c0 + 32 >= a.bt.batch) {
            const int l = m ? __ffs(m) - 1 : 31;
            k.b = min(c0 + l, a.bt.batch - 1);
            rem = at - base - __shfl_sync(0xffffffffu, v - cost, l);
            break;
        }
        base += __shfl_sync(0xffffffffu, v, 31);
    }
    k.w = SeqWork<ROWS, OV>(a, k.b);
    k.item = (int)(rem / (k.w.nblk + OV));
    k.u = (int)(rem % (k.w.nblk + OV));
    k.left = 0;
    return k;
}

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// An 8 x 8 matrix of 16-bit values held two per lane (row lane / 4), transposed.
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// c += A (16 x 16, row major) * B (16 x 8, column major)
template <class T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, f16>::value)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The exponent that probabilities are taken relative to, for scores of at most v: they may be up to 2^15 in
// fp16, so that those down to 2^-40 of the largest are still seen by the products (at 2^-25, the end with the
// largest at 1, 33000 slots 17.4 nats below it lost 9e-4 of the result while the sum counted them).  bf16 has
// fp32's range.  From 2^23 on v - 15 is too coarse for that.
template <class T>
__device__ __forceinline__ float p_top(float v) {
    return std::is_same<T, f16>::value && fabsf(v) < 8388608.0f ? v - 15.0f : v;
}

template <int C, int D, int NR>
__global__ void __launch_bounds__(DecCfg<C, D, NR>::NW * 32, 1)
    attn_rows_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    using Cfg = DecCfg<C, D, NR>;
    using T = typename CacheT<C>::Q;
    constexpr int NW = Cfg::NW, S = Cfg::S, ROWS = Cfg::ROWS, MT = D / 16;  // MT: column tiles of O^T
    constexpr int OV = dec_ov(Cfg::Q8);
    using Walk = qg::Walk<ROWS, OV>;
    extern __shared__ __align__(16) uint8_t dec_smem[];
    __shared__ int64_t sh[2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (smem_addr(dec_smem) + 1023u) & ~1023u;
    const uint32_t ring = base + (uint32_t)warp * S * 2 * Cfg::TILE;
    const uint32_t steps = base + Cfg::STEP_AT + (uint32_t)warp * S * 2 * Cfg::STEPS;
    const uint32_t bars = base + Cfg::BAR_AT + (uint32_t)warp * S * 8;
    float *merge = reinterpret_cast<float *>(dec_smem + (base - smem_addr(dec_smem)) + Cfg::MERGE_AT);
    float2 *ml = reinterpret_cast<float2 *>(dec_smem + (base - smem_addr(dec_smem)) + Cfg::ML_AT);

    if (lane == 0) {
        for (int s = 0; s < S; ++s) mbar_init(bars + 8 * s, 1);
        fence_mbar_init();
    }
    __syncwarp();
    griddep_wait();
    griddep_launch_dependents();
    int64_t total;
    int ctas;
    if (a.bt.batch <= 128) {  // every warp for itself: nobody waits
        total = walk_total<ROWS, OV>(a, ctas);
    } else {
        if (warp == 0) {
            total = walk_total<ROWS, OV>(a, ctas);
            if (lane == 0) sh[0] = total, sh[1] = ctas;
        }
        __syncthreads();
        total = sh[0], ctas = (int)sh[1];
    }
    if (tid == 0) a.desc[blockIdx.x].parts = 0;
    const Ranges rg(total, ctas);
    if ((int)blockIdx.x >= rg.ctas) return;
    const int64_t w0 = rg.start(blockIdx.x), w1 = rg.start(blockIdx.x + 1);
    if (w0 >= w1) return;
    Walk con = walk_find<ROWS, OV>(a, w0);
    con.left = w1 - w0;
    if (con.end() <= con.blk()) return;  // the range ends before the item's first block

    // ---- producer: this warp's next block, its page id fetched one block early
    Walk pro = con;
    const uint32_t mpage = (uint32_t)((0x100000000ull + a.bt.page - 1) / a.bt.page);
    int pblk = pro.blk() + warp, pend = pro.end(), ppage = 0, pslot = 0, phead = pro.item / pro.w.nrt;
    auto pro_seek = [&]() {  // moves on to a segment that has a block for this warp, and looks its page up
        while (pro.left > 0 && pblk >= pend) {
            pro.next(a);
            if (pro.left > 0) {
                pblk = pro.blk() + warp;
                pend = pro.end();
                phead = pro.item / pro.w.nrt;
            }
        }
        if (pro.left > 0) {
            const int idx = fast_div((pro.w.kb0 + pblk) * DEC_BLK, a.bt.page, mpage, pslot);
            ppage = a.bt.pages[pro.b * a.bt.table_stride + min(idx, a.bt.table_width - 1)];
        }
    };
    pro_seek();
    auto issue = [&](int s) {  // all lanes call; lane 0 copies the block into ring slot s
        if (pro.left <= 0) return;
        if (lane == 0) {
            const int slot = pslot, h = phead;
            const int page = (unsigned)ppage < (unsigned)a.bt.n_pages ? ppage : a.bt.n_pages;  // out of range: zeros
            const uint32_t kt = ring + (uint32_t)s * 2 * Cfg::TILE, vt = kt + Cfg::TILE, bar = bars + 8 * s;
            const bool st = Cfg::Q8 && page < a.bt.n_pages;
            if (Cfg::Q8 && !st) {  // no such page: steps of zero beside codes of zero
                for (int i = 0; i < 2 * Cfg::STEPS; i += 16) sts128(steps + (uint32_t)s * 2 * Cfg::STEPS + i, 0, 0, 0, 0);
            }
            mbar_arrive_expect_tx(bar, 2 * Cfg::TILE + (st ? 2 * Cfg::STEPS : 0));
#pragma unroll
            for (int p = 0; p < Cfg::NP; ++p)
                tma_load_4d(kt + p * DEC_BLK * Cfg::PANEL, &kmap, p * (Cfg::PANEL / Cfg::ES), slot, h, page, bar);
#pragma unroll
            for (int p = 0; p < Cfg::NP; ++p)
                tma_load_4d(vt + p * DEC_BLK * Cfg::PANEL, &vmap, p * (Cfg::PANEL / Cfg::ES), slot, h, page, bar);
            if (st) {
                const int64_t at = page * a.step_stride + ((int64_t)h * a.bt.page + slot) * (D / 32);
                bulk_g2s(steps + (uint32_t)s * 2 * Cfg::STEPS, a.kd + at, Cfg::STEPS, bar);
                bulk_g2s(steps + (uint32_t)(s * 2 + 1) * Cfg::STEPS, a.vd + at, Cfg::STEPS, bar);
            }
        }
        pblk += NW;
        pro_seek();
    };
    for (int s = 0; s < S; ++s) issue(s);

    const int gr = lane >> 2, gc = lane & 3;
    int slot = 0;
    uint32_t phase = 0;
    // ---- queries as B fragments: row 8 r + gr.  Beside an 8-bit cache they are kept in shared memory for all
    // warps, a lane's 8 elements of each 32-element block together: that leaves registers to the
    // conversion and lets its loop over blocks be a loop, where unrolled code misses in the
    // instruction cache
    uint32_t qf[NR][Cfg::Q8 ? 1 : MT][2];
    const uint32_t qs = base + Cfg::QS_AT + 16 * lane;
    auto load_q = [&](const Walk &k) {
        const int h = k.item / k.w.nrt, rt = k.item % k.w.nrt, nr = min(ROWS, k.w.sq.n * a.G - rt * ROWS);
        auto row = [&](int r) {  // rows past the last are copies of it: nothing of them is written
            const int rr = rt * ROWS + min(8 * r + gr, nr - 1), t = rr / a.G, g = rr % a.G;
            return static_cast<const T *>(a.q) + (int64_t)(k.w.sq.first + t) * a.ldq + (int64_t)(h * a.G + g) * a.hdq;
        };
        if constexpr (Cfg::Q8) {
            for (int x = warp; x < NR * (D / 32); x += NW) {
                const uint4 v = *reinterpret_cast<const uint4 *>(row(x / (D / 32)) + x % (D / 32) * 32 + 8 * gc);
                sts128(qs + x * 512, v.x, v.y, v.z, v.w);
            }
        } else {
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const T *src = row(r);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    qf[r][m][0] = *reinterpret_cast<const uint32_t *>(src + 16 * m + 2 * gc);
                    qf[r][m][1] = *reinterpret_cast<const uint32_t *>(src + 16 * m + 8 + 2 * gc);
                }
            }
        }
    };
    load_q(con);
    if (Cfg::Q8) __syncthreads();
    while (con.left > 0) {

        const int blk0 = con.blk(), end = con.end();
        const int h = con.item / con.w.nrt, rt = con.item % con.w.nrt;
        const Seq sq = con.w.sq;
        const int nr = min(ROWS, sq.n * a.G - rt * ROWS);
        // visible slots of the lane's rows 8 r + 2 gc, + 1
        int hi[NR][2], lo[NR][2];
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                hi[r][i] = sq.len - sq.n + (rt * ROWS + min(8 * r + 2 * gc + i, nr - 1)) / a.G;
                lo[r][i] = seen_from(hi[r][i], a.window);
            }
        const int t_first = rt * ROWS / a.G, t_last = (rt * ROWS + nr - 1) / a.G;
        const int hi_min = sq.len - sq.n + t_first;                                               // every row sees up to here
        const int lo_max = seen_from(sq.len - sq.n + t_last, a.window);                           // and from here
        const int seen_lo = seen_from(hi_min, a.window);                                          // some row sees from here
        float o[NR][MT][4];  // O^T: columns 16 m + gr, + 8 of rows 8 r + 2 gc, + 1
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[r][m][j] = 0.0f;
        float mx[NR][2], l[NR][2];
#pragma unroll
        for (int r = 0; r < NR; ++r) mx[r][0] = mx[r][1] = -INFINITY, l[r][0] = l[r][1] = 0.0f;

        for (int blk = blk0 + warp; blk < end; blk += NW) {
            const int key0 = (con.w.kb0 + blk) * DEC_BLK;
            const uint32_t kt = ring + (uint32_t)slot * 2 * Cfg::TILE, vt = kt + Cfg::TILE;
            const uint32_t ks = steps + (uint32_t)slot * 2 * Cfg::STEPS, vs = ks + Cfg::STEPS;
            mbar_wait(bars + 8 * slot, phase);
            // ---- scores: s[r][0..1] slot gr, s[r][2..3] slot gr + 8, of rows 8 r + 2 gc, + 1
            float s[NR][4] = {};
            if constexpr (!Cfg::Q8) {
                const int row = (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
                for (int k = 0; k < MT; ++k) {
                    const int ch = 2 * k + (lane >> 4);
                    uint32_t f[4];
                    ldmatrix4(kt + (ch >> 3) * DEC_BLK * 128 + row * 128 + (((ch & 7) ^ (row & 7)) << 4), f);
#pragma unroll
                    for (int r = 0; r < NR; ++r) mma16816<T>(s[r], f, qf[r][k][0], qf[r][k][1]);
                }
            } else {
                // lane (gr, gc) takes codes 8 gc .. of each 32-element block of slots gr and gr + 8
                const int half = gc >> 1, turn = Cfg::PANEL == 128 ? gr : gr >> 1;  // the rows' places in the swizzle
                const uint32_t krow = kt + gr * Cfg::PANEL + (gc & 1) * 8;
#pragma unroll 4
                for (int j = 0; j < D / 32; ++j) {
                    uint32_t f0[4], f1[4];  // codes 0..3 and 4..7 of the lane's 8, slots gr and gr + 8
                    const uint32_t at = krow + (Cfg::PANEL == 128 ? (j >> 2) * (DEC_BLK * 128) + (((2 * (j & 3) + half) ^ turn) << 4)
                                                                  : (((2 * j + half) ^ (turn & 3)) << 4));
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        uint2 v = lds64(at + n * 8 * Cfg::PANEL);
                        v.x ^= 0x80808080u;
                        v.y ^= 0x80808080u;
                        f0[n] = codes_to_f16(v.x, 0x4140);
                        f0[n + 2] = codes_to_f16(v.x, 0x4342);
                        f1[n] = codes_to_f16(v.y, 0x4140);
                        f1[n + 2] = codes_to_f16(v.y, 0x4342);
                    }
                    // the slots' steps: the codes stay exact integers in the products
                    const float d0 = half_bits_to_float(lds16(ks + (gr * (D / 32) + j) * 2));
                    const float d1 = half_bits_to_float(lds16(ks + ((gr + 8) * (D / 32) + j) * 2));
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        const uint4 q = lds128(qs + (r * (D / 32) + j) * 512);
                        float acc[4] = {};
                        mma16816<T>(acc, f0, q.x, q.y);
                        mma16816<T>(acc, f1, q.z, q.w);
                        s[r][0] = fmaf(acc[0], d0, s[r][0]);
                        s[r][1] = fmaf(acc[1], d0, s[r][1]);
                        s[r][2] = fmaf(acc[2], d1, s[r][2]);
                        s[r][3] = fmaf(acc[3], d1, s[r][3]);
                    }
                }
            }
            const bool edge = key0 + DEC_BLK - 1 > hi_min || key0 < lo_max;
            bool grown = false;
            float mn[NR][2];
#pragma unroll
            for (int r = 0; r < NR; ++r) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[r][j] *= a.scale2;
                    const int key = key0 + gr + 8 * (j >> 1), i = j & 1;
                    if (edge && (key > hi[r][i] || key < lo[r][i])) s[r][j] = -INFINITY;
                }
                // ---- running maximum over the warp's slots
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float v = fmaxf(s[r][i], s[r][2 + i]);
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                    mn[r][i] = fmaxf(mx[r][i], p_top<T>(v));
                    grown = grown || mn[r][i] > mx[r][i];
                }
            }
            if (__any_sync(0xffffffffu, grown)) {  // the sums are rescaled only where it grew
#pragma unroll
                for (int r = 0; r < NR; ++r)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float f = mn[r][i] > mx[r][i] ? exp2_approx(mx[r][i] - mn[r][i]) : 1.0f;  // mx = -inf: 0
                        mx[r][i] = mn[r][i];
                        l[r][i] *= f;
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            o[r][m][i] *= f;
                            o[r][m][2 + i] *= f;
                        }
                    }
            }
            uint32_t ph[NR][2], pl[NR][2];  // probabilities as B fragments, hi + lo
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const float z0 = mx[r][0] == -INFINITY ? 0.0f : mx[r][0], z1 = mx[r][1] == -INFINITY ? 0.0f : mx[r][1];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float p0 = exp2_approx(s[r][2 * n] - z0), p1 = exp2_approx(s[r][2 * n + 1] - z1);
                    l[r][0] += p0;
                    l[r][1] += p1;
                    const uint32_t hb = pack2<T>(p0, p1);
                    const float2 hf = unpack2<T>(hb);
                    ph[r][n] = movmatrix_t(hb);
                    pl[r][n] = movmatrix_t(pack2<T>(p0 - hf.x, p1 - hf.y));
                }
            }
            // slots that no row sees may hold anything: their values (the steps of their codes) become zeros
            if (key0 + DEC_BLK > sq.len || key0 < seen_lo) {
                constexpr int RB = Cfg::Q8 ? D / 32 * 2 : Cfg::PANEL;  // bytes of a row in one place
                constexpr int PL = Cfg::Q8 ? 1 : Cfg::NP;
                for (int x = lane; x < DEC_BLK * PL * (RB / 4); x += 32) {
                    const int row = x / (RB / 4) % DEC_BLK, key = key0 + row;
                    if (key >= sq.len || key < seen_lo) sts32((Cfg::Q8 ? vs : vt) + 4 * x, 0u);
                }
                __syncwarp();
            }
            if constexpr (!Cfg::Q8) {
                const int row = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const int ch = 2 * m + ((lane >> 3) & 1);
                    uint32_t f[4];
                    ldmatrix4_t(vt + (ch >> 3) * DEC_BLK * 128 + row * 128 + (((ch & 7) ^ (row & 7)) << 4), f);
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        mma16816<T>(o[r][m], f, ph[r][0], ph[r][1]);
                        mma16816<T>(o[r][m], f, pl[r][0], pl[r][1]);
                    }
                }
            } else {
                // lane (gr, gc) reads the codes gr * EPR .. of slots 2 gc, 2 gc + 1, 2 gc + 8, 2 gc + 9 in
                // each panel: product i then covers columns gr * EPR + 2 i (first 8 rows of the tile) and + 1
                constexpr int EPR = Cfg::PANEL / 8;  // 16, or 8 where rows are 64 bytes
#pragma unroll
                for (int p = 0; p < Cfg::NP; ++p) {
                    uint32_t w[4][EPR / 4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int row = 2 * gc + (q & 1) + 8 * (q >> 1);
                        if constexpr (EPR == 16) {
                            const uint4 v = lds128(vt + p * DEC_BLK * 128 + row * 128 + ((gr ^ (row & 7)) << 4));
                            w[q][0] = v.x, w[q][1] = v.y, w[q][2] = v.z, w[q][3] = v.w;
                        } else {
                            const uint2 v = lds64(vt + row * 64 + (((gr >> 1) ^ ((row >> 1) & 3)) << 4) + (gr & 1) * 8);
                            w[q][0] = v.x, w[q][1] = v.y;
                        }
#pragma unroll
                        for (int e = 0; e < EPR / 4; ++e) w[q][e] ^= 0x80808080u;
                    }
                    // the steps of those slots for the 32-element block that holds the lane's columns
                    const int j = (p * 128 + gr * EPR) >> 5;
                    __half2 d[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t at = vs + ((2 * gc + 8 * i) * (D / 32) + j) * 2;
                        const uint32_t b = lds16(at) | lds16(at + (D / 32) * 2) << 16;
                        d[i] = *reinterpret_cast<const __half2 *>(&b);
                    }
#pragma unroll
                    for (int e = 0; e < EPR / 4; ++e) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {  // bytes 2 x and 2 x + 1 of the words
                            uint32_t f[4];
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                // (a0, b0, a1, b1) of two slots' bytes, then each pair under 0x64
                                const uint32_t two = prmt(w[2 * i][e], w[2 * i + 1][e], x ? 0x7362u : 0x5140u);
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    const uint32_t c = codes_to_f16(two, y ? 0x4342 : 0x4140);
                                    const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&c), d[i]);
                                    f[2 * i + y] = *reinterpret_cast<const uint32_t *>(&v);
                                }
                            }
                            const int m = p * (EPR / 2) + 2 * e + x;
#pragma unroll
                            for (int r = 0; r < NR; ++r) {
                                mma16816<T>(o[r][m], f, ph[r][0], ph[r][1]);
                                mma16816<T>(o[r][m], f, pl[r][0], pl[r][1]);
                            }
                        }
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();  // every lane has read the slot
            issue(slot);
            if (++slot == S) {
                slot = 0;
                phase ^= 1;
            }
        }

        // ---- merge the warps' results; the next item's queries come in meanwhile
        Walk nxt = con;
        nxt.next(a);
        if (!Cfg::Q8 && nxt.left > 0) load_q(nxt);
        const bool whole = blk0 == 0 && end == con.w.nblk;
        if (warp == 0 && blk0 == 0 && !whole) {
            const int64_t s0 = w1 - con.left - con.u;  // the item's first unit
            const int parts = rg.parts(blockIdx.x, s0 + con.w.nblk + OV);
            if (lane == 0) a.desc[blockIdx.x] = JoinDesc{parts, sq.first, h, rt * ROWS, sq.n * a.G, {}};
        }
        float f[NR][2];
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l[r][i] += __shfl_xor_sync(0xffffffffu, l[r][i], 4);
                l[r][i] += __shfl_xor_sync(0xffffffffu, l[r][i], 8);
                l[r][i] += __shfl_xor_sync(0xffffffffu, l[r][i], 16);
                if (gr == 0) ml[warp * ROWS + 8 * r + 2 * gc + i] = make_float2(mx[r][i], l[r][i]);
            }
        __syncthreads();  // every warp has left the item's slots
        if (Cfg::Q8 && nxt.left > 0) load_q(nxt);  // before the merge's last barrier
        float *part = a.part + (size_t)(2 * blockIdx.x + (blk0 == 0 ? 1 : 0)) * attn_part_floats(ROWS, D);
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = 8 * r + 2 * gc + i;
                float top = -INFINITY, sum = 0.0f;
#pragma unroll
                for (int w = 0; w < NW; ++w) top = fmaxf(top, ml[w * ROWS + row].x);
                const float z = top == -INFINITY ? 0.0f : top;
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    const float2 v = ml[w * ROWS + row];
                    sum += v.y * exp2_approx(v.x - z);
                }
                f[r][i] = sum > 0.0f ? exp2_approx(mx[r][i] - z) / sum : 0.0f;
                if (sum != sum) f[r][i] = sum;  // a NaN score stays one
                if (warp == 0 && gr == 0 && row < nr) {
                    const float ls = sum > 0.0f ? z + log2_approx(sum) : sum == 0.0f ? -INFINITY : sum;
                    const int rr = rt * ROWS + row;
                    if (!whole)
                        part[ROWS * D + row] = ls;
                    else if (a.lse)
                        a.lse[(int64_t)(sq.first + rr / a.G) * a.Hq + h * a.G + rr % a.G] = ls * LN2;
                }
            }
        // MW columns at a time: [warp][row][MW]
        constexpr int MW = Cfg::MW;
#pragma unroll
        for (int c0 = 0; c0 < MT; c0 += MW / 16) {
            if (c0) __syncthreads();
#pragma unroll
            for (int m = 0; m < MW / 16; ++m)
#pragma unroll
                for (int r = 0; r < NR; ++r)
#pragma unroll
                    for (int j = 0; j < 4; ++j)  // place 16 m + 8 (j / 2) + gr: tile c0 + m, its row gr or gr + 8
                        merge[(warp * ROWS + 8 * r + 2 * gc + (j & 1)) * MW + ((16 * m + 8 * (j >> 1) + gr) ^ (8 * gc))] =
                            o[r][c0 + m][j] * f[r][j & 1];
            __syncthreads();
            for (int x = tid; x < nr * MW; x += NW * 32) {
                const int r = x / MW, j = x % MW;
                float v = 0.0f;
#pragma unroll
                for (int w = 0; w < NW; ++w) v += merge[(w * ROWS + r) * MW + (j ^ (8 * ((r >> 1) & 3)))];
                const int m = c0 + j / 16, e = j & 15;
                int col;
                if constexpr (!Cfg::Q8) {
                    col = 16 * m + e;
                } else {
                    constexpr int EPR = Cfg::PANEL / 8;
                    col = (m / (EPR / 2)) * Cfg::PANEL + (e & 7) * EPR + 2 * (m % (EPR / 2)) + (e >> 3);
                }
                const int rr = rt * ROWS + r;
                if (!whole) {
                    part[r * D + col] = v;
                } else {
                    const int64_t at = ((int64_t)(sq.first + rr / a.G) * a.Hq + h * a.G + rr % a.G) * D + col;
                    if (a.out_f32)
                        static_cast<float *>(a.out)[at] = v;
                    else
                        static_cast<T *>(a.out)[at] = from_f32<T>(v);
                }
            }
        }
        __syncthreads();  // ml and merge are free again
        con = nxt;
    }
    // every copy that was issued has been waited for, unless a wait gave up: let those land
    for (int s = 0; s < S; ++s)
        if (lane == 0) mbar_drain(bars + 8 * s, (s < slot ? phase : phase ^ 1), DRAIN_NS);
}

// Merges the partial results of the items that range boundaries cut, and clears the rows of tokens that belong to no
// sequence (the last x: the last CTA leaves no item to others).  Block (x, y): the item that
// CTA x described, its row y.  Partial i carries weight 2^(lse_i - max); the warps take every
// JOIN_WARPS-th partial.
constexpr int JOIN_WARPS = 8;
constexpr int JOIN_MAX = 1024;  // ranges (SMs) at most

template <class T, int D, int NR>
__global__ void __launch_bounds__(JOIN_WARPS * 32) attn_join_kernel(const AttnArgs a) {
    constexpr int ROWS = 8 * NR, V = D / 32;
    __shared__ float wt[JOIN_MAX], red[JOIN_WARPS], acc[JOIN_WARPS][D];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = blockIdx.y;
    if (blockIdx.x == gridDim.x - 1) {
        clear_outside<T>(a, D);
        return;
    }
    const JoinDesc jd = a.desc[blockIdx.x];
    const int parts = jd.parts, rr = jd.row0 + r;
    if (parts == 0 || rr >= jd.nrows) return;
    auto part = [&](int i) {  // the item ends the first range and starts the others
        return a.part + (size_t)(2 * ((int)blockIdx.x + i) + (i == 0 ? 1 : 0)) * attn_part_floats(ROWS, D);
    };
    float mx = -INFINITY;
    for (int i = tid; i < parts; i += JOIN_WARPS * 32) mx = fmaxf(mx, wt[i] = part(i)[ROWS * D + r]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (lane == 0) red[warp] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < JOIN_WARPS; ++w) mx = fmaxf(mx, red[w]);
    const float mz = mx == -INFINITY ? 0.0f : mx;
    float sum = 0.0f, v[V] = {};
#pragma unroll 4
    for (int i = warp; i < parts; i += JOIN_WARPS) {
        float x[V];
        load_vec<float, V>(part(i) + r * D + lane * V, x);
        const float w = exp2_approx(wt[i] - mz);
        sum += w;
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = fmaf(w, x[e], v[e]);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) acc[warp][lane * V + e] = v[e];
    __syncthreads();  // red has been read
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < JOIN_WARPS; ++w) sum += red[w];
    const int64_t row = (int64_t)(jd.first + rr / a.G) * a.Hq + jd.h * a.G + rr % a.G;
    for (int c = tid; c < D; c += JOIN_WARPS * 32) {
        float x = 0.0f;
#pragma unroll
        for (int w = 0; w < JOIN_WARPS; ++w) x += acc[w][c];
        x = sum > 0.0f ? x / sum : sum;
        if (a.out_f32)
            static_cast<float *>(a.out)[row * D + c] = x;
        else
            static_cast<T *>(a.out)[row * D + c] = from_f32<T>(x);
    }
    if (a.lse && tid == 0) a.lse[row] = sum > 0.0f ? (mz + log2_approx(sum)) * LN2 : sum == 0.0f ? -INFINITY : sum;
}

// ----------------------------------------------------------------------------- host
// Dynamic shared memory above 48 KB is asked for once per kernel and device.
bool allow_smem(const void *kern, uint32_t bytes) {
    static std::mutex mu;
    static std::set<std::pair<const void *, int>> done;
    return once_per_device(done, mu, kern,
                           [&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess; });
}

typedef CUresult (*PFN_encode_tiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                     const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                     CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static PFN_encode_tiled encode_tiled() {
    static const PFN_encode_tiled encode = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            f = nullptr;
        }
        return reinterpret_cast<PFN_encode_tiled>(f);
    }();
    return encode;
}

bool attn_query_map(CUtensorMap *map, const AttnArgs &a, bool is_bf16, int D) {
    const PFN_encode_tiled encode = encode_tiled();
    if (!encode) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)a.G, (cuuint64_t)a.Hk, (cuuint64_t)a.bt.tokens};
    const cuuint64_t strides[3] = {(cuuint64_t)a.hdq * 2, (cuuint64_t)a.hdq * 2 * a.G, (cuuint64_t)a.ldq * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)a.G, 1, (cuuint32_t)(128 / a.G)};
    const cuuint32_t unit[4] = {1, 1, 1, 1};
    return encode(map, is_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void *>(a.q), dims, strides,
                  box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool attn_tensor_map(CUtensorMap *map, const qg_paged &c, const void *base, int rows) {
    const PFN_encode_tiled encode = encode_tiled();
    if (!encode) return false;
    const int es = c.type == QG_Q8_0 ? 1 : 2, row = c.dim * es;
    const cuuint64_t dims[4] = {(cuuint64_t)c.dim, (cuuint64_t)c.page, (cuuint64_t)c.kv_heads, (cuuint64_t)c.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.slot_stride * es, (cuuint64_t)c.head_stride * es, (cuuint64_t)c.page_stride * es};
    const cuuint32_t box[4] = {(cuuint32_t)(std::min(row, 128) / es), (cuuint32_t)rows, 1, 1};
    const cuuint32_t unit[4] = {1, 1, 1, 1};
    const CUtensorMapDataType type = c.type == QG_Q8_0   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : c.type == QG_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                          : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return encode(map, type, 4, const_cast<void *>(base), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  row >= 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int C, int D, int NR>
static int attn_rows_run(const AttnArgs &a, const qg_paged &c, int sms, cudaStream_t s) {
    using Cfg = DecCfg<C, D, NR>;
    static_assert(Cfg::BYTES <= SMEM_MAX, "shared memory of the row kernel");
    CUtensorMap km, vm;
    if (!attn_tensor_map(&km, c, c.k, DEC_BLK) || !attn_tensor_map(&vm, c, c.v, DEC_BLK)) return QG_ECUDA;
    auto kern = attn_rows_kernel<C, D, NR>;
    if (!allow_smem((const void *)kern, Cfg::BYTES)) return QG_ECUDA;
    const int ctas = std::min(sms, JOIN_MAX);
    if (!launch_programmatic(kern, dim3((unsigned)ctas), Cfg::NW * 32, Cfg::BYTES, s, a, km, vm)) return QG_ECUDA;
    const int rows = (int)std::min<int64_t>(Cfg::ROWS, (int64_t)a.bt.tokens * a.G);
    auto join = attn_join_kernel<typename CacheT<C>::Q, D, NR>;
    return launch_programmatic(join, dim3((unsigned)ctas, (unsigned)rows), JOIN_WARPS * 32, 0, s, a) ? QG_OK : QG_ECUDA;
}
template <int C, int NR>
static int attn_rows_dim(const AttnArgs &a, const qg_paged &c, int sms, cudaStream_t s) {
    return c.dim == 64    ? attn_rows_run<C, 64, NR>(a, c, sms, s)
           : c.dim == 128 ? attn_rows_run<C, 128, NR>(a, c, sms, s)
                          : attn_rows_run<C, 256, NR>(a, c, sms, s);
}
template <int NR>
static int attn_rows(const AttnArgs &a, const qg_paged &c, int sms, cudaStream_t s) {
    return c.type == QG_F16    ? attn_rows_dim<CACHE_F16, NR>(a, c, sms, s)
           : c.type == QG_BF16 ? attn_rows_dim<CACHE_BF16, NR>(a, c, sms, s)
                               : attn_rows_dim<CACHE_Q8, NR>(a, c, sms, s);
}

int attn_dev_err_take(unsigned int *err) {
    unsigned int zero = 0;
    if (cudaMemcpyFromSymbol(err, g_qg_dev_err, sizeof(*err)) != cudaSuccess) return QG_ECUDA;
    if (cudaMemcpyToSymbol(g_qg_dev_err, &zero, sizeof(zero)) != cudaSuccess) return QG_ECUDA;
    unsigned int more = 0;
    const int rc = attn_chunk_dev_err_take(&more);
    *err |= more;
    return rc;
}

}  // namespace qg

using namespace qg;

extern "C" {

size_t qg_attn_workspace_size(int dim, int q_heads, int kv_heads, int tokens, int batch) {
    if ((dim != 64 && dim != 128 && dim != 256) || kv_heads < 1 || q_heads < 1 || q_heads % kv_heads || tokens < 1 || batch < 1)
        return (size_t)-1;
    const int sms = device_sms_planning();
    const size_t rows = (size_t)sms * 2 * attn_part_floats(DEC_ROWS, dim) * sizeof(float);
    return (size_t)sms * sizeof(JoinDesc) + std::max(rows, attn_chunk_workspace(dim, q_heads / kv_heads, tokens, batch, sms));
}

int qg_attn_paged(const void *q, int64_t ldq, int64_t hdq, int q_type, int tokens, int q_heads, int max_new, float scale,
                  int window, void *out, int out_type, float *lse, const qg_paged *cache, void *ws, size_t ws_bytes,
                  void *stream) {
    if (!q || !out || !cache || tokens < 1 || q_heads < 1 || max_new < 0 || window < 0 || !(scale == scale)) return QG_EINVAL;
    if (const int rc = paged_check(*cache)) return rc;
    if (q_type != (cache->type == QG_BF16 ? QG_BF16 : QG_F16) || (out_type != q_type && out_type != QG_F32)) return QG_EINVAL;
    const int D = cache->dim;
    if (q_heads % cache->kv_heads || ldq < D || hdq < D) return QG_EINVAL;
    if ((int64_t)tokens * q_heads > INT32_MAX) return QG_EINVAL;  // rows of out are counted in 32 bits
    if (!host_aligned(q, 16) || ldq % 8 || hdq % 8 || !host_aligned(out, 16) || !host_aligned(lse, 4)) return QG_EALIGN;
    if (!ws || ws_bytes < qg_attn_workspace_size(D, q_heads, cache->kv_heads, tokens, cache->batch)) return QG_EWORKSPACE;
    if (!host_aligned(ws, 16)) return QG_EALIGN;
    const int sms = device_sms();
    if (sms < 0) return sms;
    AttnArgs a{};
    a.bt = paged_batch(*cache, tokens);
    a.q = q, a.ldq = ldq, a.hdq = hdq;
    a.out = out, a.lse = lse;
    a.Hq = q_heads, a.Hk = cache->kv_heads, a.G = q_heads / cache->kv_heads;
    a.out_f32 = out_type == QG_F32;
    a.window = window;
    a.scale2 = scale * LOG2E;
    a.kd = static_cast<const f16 *>(cache->kd), a.vd = static_cast<const f16 *>(cache->vd);
    a.step_stride = cache->step_stride;
    a.desc = static_cast<JoinDesc *>(ws);
    a.part = reinterpret_cast<float *>(a.desc + sms);
    cudaStream_t s = (cudaStream_t)stream;
    // one row tile of 16 per sequence and cache head: the row kernel reads the cache once
    if ((int64_t)max_new * a.G > DEC_ROWS) return attn_chunk(a, *cache, sms, s);
    return (int64_t)max_new * a.G <= 8 ? attn_rows<1>(a, *cache, sms, s) : attn_rows<2>(a, *cache, sms, s);
}

}  // extern "C"
