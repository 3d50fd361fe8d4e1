// qg_chunk.cu -- attention of chunks of new tokens over a paged cache on the 5th-generation tensor
// cores: the plan of the row tiles, the kernel, and the merge of items that were cut.
//
// Row r of a sequence is query head g = r % G of a cache head and new token r / G, so the G heads
// that share a cache head share each slot's copy.  A CTA multiplies NQ tiles of 128 rows with tiles
// of BN slots:
//   * producer: one warp copies the key and value tiles through the page table, a tiled TMA copy
//     per page and 128-byte panel (pages end inside a tile); from 8-bit caches it copies codes and
//     steps, which one or two more warpgroups turn into tiles of step * code in fp16;
//   * MMA warp: scores S = Q K^T (128 x BN, fp32 in tensor memory), then O += P V;
//   * a warpgroup per row tile: each thread owns one row, so its maximum and sum need no
//     exchange (the running maximum and sum are those of Milakov and Gimelshein, Online normalizer
//     calculation for softmax, 2018, here rescaled only now and then); it reads S, writes P = 2^(S - m) and, where the maximum has grown by more than
//     2^8, rescales O.  Up to there a stale maximum is as good: O and the sum carry the same
//     factor.  In fp16 P is 2^(S - m + 7), at most 2^15: slots down to 2^-32 of the largest are
//     seen by the products, where at 2^-25 a long flat tail was lost that the sum counted.
// What a row tile's warpgroup does for one slot tile (read S, maximum, exponentials, write P) takes
// about as long as the tile's two products with their latencies, so the next scores have to run
// under it: a score buffer is free again as soon as its rows are in registers, as P has columns of
// its own.  Tensor memory (512 columns) holds two score buffers, two P and two O at dim 64; at
// dim 128 one score buffer on which the row tiles take turns; at dim 256, whose O fills half of it,
// one row tile with two score buffers, P over its scores.  The value product starts on the first
// half of P while the second is made.  Measured and dropped for dim 128 (4096 tokens after 28000,
// 32/8 heads, bf16): P over its scores and a score buffer per row tile, so that a tile's scores
// wait for its last value product, 1.98 ms; P in shared memory, whose bandwidth then is the bound,
// 1.83 ms; now 1.52 ms (1.33 PFLOP/s).  No product relies on the order of another that writes different columns:
// each waits for the barrier of what it overwrites, and each row tile's products are issued by a
// warp of their own.
// P is rounded to the value's 16-bit type, the operand type of the product: one rounding of
// relative size 2^-12 (2^-9) per factor on average beside that of the result.  8-bit keys and values
// become fp16 operands, step * code rounded once (relative 2^-12): the tensor cores take no int8
// beside fp16, and splitting the step off would need a product per block of 32.
//
// The roles run at once and their code shares the instruction cache, which is what a kernel with
// converting warps is sensitive to: each role's loop is written once and left rolled (softmax in chunks of
// 32 scores, one place for all copies, one for each product).  512 tokens after 8000, 24/4 heads of 256,
// 8-bit: 194 us with the roles unrolled, 146 now (0.71 PFLOP/s); there the conversion and the chain scores ->
// softmax -> values of the single row tile take about equally long, and neither hides the other
// entirely.  512 after 8000 of 32/8 heads, 8-bit: 77 us at dim 64, 128 at 128, where one converting warpgroup
// feeds two row tiles and the softmax reads its scores twice (16-bit: 55 and 71; 131 at dim 256 against
// 179).  With two row tiles and 16-bit caches the tensor cores are the bound for long chunks, the
// exponentials (16 a clock and SM) at dim 64.
//
// Work is counted in slot tiles over all items (row tile, cache head).  Where dealing whole items out,
// the largest first and back and forth over the CTAs, loads them evenly enough, that is done: no
// partial results, nothing to merge.  Else the list is cut into one equal range per CTA, so that
// ragged batches and a few rows over a long context load the machine evenly too.
#include <algorithm>
#include <cmath>
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
    static constexpr int BN = 128;
    static constexpr int ROWS = NQ * 128;
    static constexpr int NP = D / 64;            // 128-byte panels of a row
    // A slot tile's keys are copied in KU units of whole panels, its values in as many of whole rows
    static constexpr int KU = D == 256 ? 2 : 1;
    static constexpr int PKU = NP / KU;          // panels of a key unit
    static constexpr int VR = BN / KU;           // rows of a value unit
    static constexpr int NS = D == 64 ? 6 : Q8 ? 3 : 4;  // units in shared memory
    static constexpr uint32_t QB = 128 * D * 2;
    static constexpr uint32_t TILE = BN * D * 2 / KU;
    // P goes over the scores it came from where two score buffers alternate (dim 256), else beside them;
    // with dim 128 the row tiles take turns on one score buffer
    static constexpr bool P_OVER = D == 256, S_TURNS = D == 128;
    static constexpr int S_COLS = S_TURNS ? BN : NQ * SB * BN;
    // 8-bit units as copied: NRAW areas of codes in swizzled rows of a panel each, then the steps of their rows
    static constexpr int NRAW = D == 128 ? 2 : 3;
    static constexpr uint32_t CODES = BN * D / KU, STEPS = BN * (D / 32) * 2;
    static constexpr int CPANEL = D < 128 ? D : 128, KCP = CODES / (BN * CPANEL), VCP = CODES / (VR * CPANEL);
    // Warpgroups: one per row tile, one whose first warps issue each row tile's products and the copies,
    // and those that convert 8-bit codes
    static constexpr int MMA_WARP = 4 * NQ;
    static constexpr int CONV_WARP = MMA_WARP + 4;
    static constexpr int NCONV = !Q8 ? 0 : D == 256 ? 2 : 1;  // unit u is converted by warpgroup u % NCONV
    static constexpr int WGS = NQ + 1 + NCONV;
    static constexpr int THREADS = WGS * 128;
    // Registers per thread at launch, and where each kind of warpgroup goes from there (0: stays).
    // Their sums are the same, so every increase is met by a decrease.
    static constexpr int LAUNCH_REGS = WGS == 2 ? 255 : WGS == 3 ? 168 : 128;
    static constexpr int ROW_REGS = WGS == 2 ? 0 : !Q8 ? 208 : NQ == 2 ? 152 : 208;
    static constexpr int ISSUE_REGS = WGS == 2 ? 0 : !Q8 ? 88 : NQ == 2 ? 72 : 64;
    static constexpr int CONV_REGS = !Q8 ? 0 : NQ == 2 ? 136 : 120;
    static_assert(WGS == 2 || NQ * ROW_REGS + ISSUE_REGS + NCONV * CONV_REGS == WGS * LAUNCH_REGS, "registers");
    // A row's scores stay in a thread's registers, all code unrolled, where two row tiles' warps run the
    // same code (4096 tokens after 28000, dim 128: 1.53 ms; in short loops 2.7).  With one row tile, or
    // converting warps beside it, two passes of 32 scores at a time in short loops are faster, as the roles then
    // share the instruction cache: 512 tokens after 8000, dim 256, 8-bit 194 -> 168 us, fp16 140 -> 128
    static constexpr bool HOLD = !Q8 && D != 256;
    static_assert(!(HOLD && P_OVER), "scores in registers free their buffer at once");
    static constexpr float P_SHIFT = C == CACHE_BF16 ? 0.0f : 7.0f;  // base-2 exponent that P has more
    // Every converting warpgroup has its own barriers for copied codes, one per area (raw_bar)
    static constexpr int NRAWBAR = NRAW * (NCONV > 1 ? NCONV : 1);
    static constexpr int NBAR = 2 * NS + 2 * NQ + 4 * NQ * SB + 1 + NRAW + NRAWBAR;
    static constexpr uint32_t OUT_AT = NQ * QB;  // 32 rows x 64 bytes of results per warp
    static constexpr uint32_t KV_AT = OUT_AT + NQ * 4 * 2048;
    static constexpr uint32_t RAW_AT = KV_AT + NS * TILE;
    static constexpr uint32_t BAR_AT = RAW_AT + (Q8 ? NRAW * (CODES + STEPS) : 0);
    static constexpr uint32_t BYTES = BAR_AT + NBAR * 8 + 8 /* tensor memory address, turn */ + 1024 /* alignment */;
    static_assert(OUT_AT % 1024 == 0 && KV_AT % 1024 == 0 && RAW_AT % 1024 == 0 && BAR_AT % 16 == 0 && TILE % 1024 == 0 && CODES % 1024 == 0 &&
                      STEPS % 16 == 0,
                  "alignment");
    // tensor memory columns
    static constexpr int O_COL = S_COLS;
    static constexpr int P_COL = O_COL + NQ * D;  // where P has columns of its own
    static constexpr int COLS = 512;
    static_assert(P_COL + (P_OVER ? 0 : NQ * BN / 2) <= COLS, "tensor memory");
};

// ----------------------------------------------------------------------------- plan
struct ChunkTile {
    int b, row0, kb0, nt;     // sequence, first row, first slot tile, slot tiles (at least 1)
    int first, n, len, pad;   // Seq of b
};
struct ChunkPlan {
    int64_t *total;    // tiles of all items
    int *nrt;          // row tiles
    int *dealt;        // whole items are dealt out: the tiles are in order of falling cost
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
    c.dealt = reinterpret_cast<int *>(p + 12);
    c.tile = reinterpret_cast<ChunkTile *>(p + 16);
    c.prefix = reinterpret_cast<int64_t *>(p + 16 + (size_t)tiles * sizeof(ChunkTile));
    return c;
}

constexpr int PLAN_THREADS = 256, PLAN_SEQS = 1024;

// An item costs its slot tiles and CHUNK_OV more for loading the queries and writing the result, in
// the same unit; a range that ends inside that part leaves the item to the next CTA.  Measured with 1,
// 3, 4: 40 sequences of about 20 new tokens, 32/8 heads of 128, fp16 75, 71, 69 us; 512 tokens after 8000,
// 24/4 heads of 256, 8-bit 144, 146, 149.  A cut is worth CHUNK_CUT: with 2 instead of 4 or 8 the mixed
// batch (12 sequences, heads of 64, window 1024) takes 34 us instead of 29.5.
constexpr int CHUNK_OV = 3;
constexpr int CHUNK_CUT = 4;        // what a cut costs a CTA: a partial result more, and its merge
constexpr int CHUNK_MIN_UNITS = 4;  // a CTA takes at least

// The k-th item of CTA c where whole items are dealt out back and forth.
__device__ __forceinline__ int deal(int k, int c, int ctas) { return k & 1 ? (k + 1) * ctas - 1 - c : k * ctas + c; }

// One block lists the row tiles of all sequences with their slot ranges.  It stands before the
// attention kernel in time, so it is built for few steps: one warp places the sequences' first tiles,
// then a thread makes a tile and one barrier a prefix of their costs.
__global__ void __launch_bounds__(PLAN_THREADS) attn_plan_kernel(const AttnArgs a, ChunkPlan p, int rows, int bn, int max_tiles, int ctas) {
    __shared__ int64_t part[2][PLAN_THREADS / 32];
    __shared__ int unit[PLAN_THREADS], sorted[PLAN_THREADS];
    __shared__ int off[PLAN_SEQS + 1];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int64_t cost_before = 0;
    int tiles_before = 0, flip = 0, dealt = 0;
    for (int c0 = 0; c0 < a.bt.batch; c0 += PLAN_SEQS) {
        const int nb = min(PLAN_SEQS, a.bt.batch - c0);
        if (c0) __syncthreads();
        if (warp == 0) {
            int before = 0;
            for (int b0 = 0; b0 < nb; b0 += 32) {
                int v = b0 + lane < nb ? (seq_of(a.bt, c0 + b0 + lane).n * a.G + rows - 1) / rows : 0;
                // q_start that decreases could list more tiles than the call's tokens make: counts stop there, and
                // those past it are left out
                v = min(v, max_tiles);
                const int mine = v;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int u = __shfl_up_sync(0xffffffffu, v, o);
                    if (lane >= o) v += u;
                }
                if (b0 + lane < nb) off[b0 + lane] = min(before + v - mine, max_tiles);
                before = min(before + __shfl_sync(0xffffffffu, v, 31), max_tiles);
            }
            if (lane == 0) off[nb] = before;
        }
        __syncthreads();
        const int count = min(off[nb], max_tiles - tiles_before);
        for (int r0 = 0; r0 < count; r0 += PLAN_THREADS) {
            const int r = r0 + tid, at = tiles_before + r;
            int64_t cost = 0;
            ChunkTile t{};
            const bool on = r < count;
            if (on) {
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
                const int from = seen_from(s.len - s.n + tf, a.window);
                const int end = s.len - s.n + tl + 1;  // slots that the last row sees
                t.kb0 = from / bn;
                t.nt = max(1, (end + bn - 1) / bn - t.kb0);
                cost = (int64_t)(t.nt + CHUNK_OV) * a.Hk;
            }
            int64_t v = cost;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            if (lane == 31) part[flip][warp] = v;
            __syncthreads();
            int64_t sum = 0;
#pragma unroll
            for (int w = 0; w < PLAN_THREADS / 32; ++w) {
                if (w == warp) v += sum;
                sum += part[flip][w];
            }
            // A single round of tiles: order them by falling cost and see how evenly whole items load the CTAs
            int place = at;
            if (a.bt.batch <= PLAN_SEQS && count <= PLAN_THREADS) {
                const int mine = on ? t.nt + CHUNK_OV : 0;
                unit[tid] = mine;
                __syncthreads();
                int rank = 0;
#pragma unroll 8
                for (int i = 0; i < count; ++i) rank += unit[i] > mine || (unit[i] == mine && i < tid);
                if (on) sorted[rank] = mine;
                __syncthreads();
                const int items = count * a.Hk;
                int64_t most = 0;
                for (int c = tid; c < ctas; c += PLAN_THREADS) {
                    int64_t load = 0;
                    for (int k = 0, i = c; i < items; ++k, i = deal(k, c, ctas)) load += sorted[i / a.Hk];
                    most = max(most, load);
                }
                dealt = !__syncthreads_or((most - CHUNK_CUT) * ctas > sum);
                if (dealt) place = rank;
            }
            if (on) {
                p.tile[place] = t;
                p.prefix[at] = cost_before + v - cost;
            }
            cost_before += sum;
            flip ^= 1;
        }
        tiles_before += count;
    }
    if (tid == 0) {
        *p.total = cost_before;
        *p.nrt = tiles_before;
        *p.dealt = dealt;
    }
}

// Position in the work list: every role of a CTA walks it by itself.
struct ChunkWalk {
    ChunkTile t;
    int rt, h, u;  // row tile, cache head, unit of the item
    int64_t left;  // units left in this CTA's range (of the item, where items are dealt out)
    int turn;      // items dealt to this CTA before
    __device__ __forceinline__ int blk() const { return max(0, u - CHUNK_OV); }  // first slot tile of the segment
    __device__ __forceinline__ int end() const { return (int)min((int64_t)t.nt, max((int64_t)0, u + left - CHUNK_OV)); }
};
__device__ __forceinline__ ChunkTile chunk_tile(const ChunkPlan &p, int rt) {
    const int4 x = reinterpret_cast<const int4 *>(p.tile + rt)[0], y = reinterpret_cast<const int4 *>(p.tile + rt)[1];
    return ChunkTile{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
}
// The position of unit `at` of the list; whole warp.
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
    k.h = (int)(rem / (k.t.nt + CHUNK_OV));
    k.u = (int)(rem % (k.t.nt + CHUNK_OV));
    k.left = 0;
    k.turn = 0;
    return k;
}
// The item of turn k.turn of this CTA out of `dealt` items; left is 0 where there is none.
__device__ __forceinline__ void chunk_deal(ChunkWalk &k, const ChunkPlan &p, int Hk, int dealt) {
    const int i = deal(k.turn, blockIdx.x, gridDim.x);
    k.left = 0;
    if (i >= dealt) return;
    k.rt = i / Hk;
    k.h = i % Hk;
    k.t = chunk_tile(p, k.rt);
    k.u = CHUNK_OV;
    k.left = k.t.nt;
}
// On to the next item of the range, or of those dealt (dealt: how many, 0: ranges); left is 0 at the end.
__device__ __forceinline__ void chunk_next(ChunkWalk &k, const ChunkPlan &p, int Hk, int dealt) {
    if (dealt) {
        ++k.turn;
        chunk_deal(k, p, Hk, dealt);
        return;
    }
    k.left -= k.t.nt + CHUNK_OV - k.u;
    k.u = 0;
    // a rest of CHUNK_OV units or less holds no slot tile
    if (k.left <= CHUNK_OV) {
        k.left = 0;
        return;
    }
    if (++k.h < Hk) return;
    k.h = 0;
    k.t = chunk_tile(p, ++k.rt);
}
__device__ __forceinline__ int chunk_ctas(int64_t total, int max_ctas) {
    return (int)min((int64_t)max_ctas, max((int64_t)1, total / CHUNK_MIN_UNITS));
}

// Whether a row's scaled maximum is so large that S * scale2 - m * scale2 is not near 0 at S = m any more: the
// product with m is rounded to a multiple of 1/2 and more.  The factor is a power of two then, whose products
// are exact; the scores themselves are off by more than what that changes.
__device__ __forceinline__ bool chunk_far(float m, float scale2) { return !(fabsf(m * scale2) < 4194304.0f); }

// ----------------------------------------------------------------------------- kernel
template <int C, int D>
__global__ void __launch_bounds__(ChunkCfg<C, D>::THREADS, 1)
    attn_chunk_kernel(const AttnArgs a, const ChunkPlan plan, int box_rows, uint32_t qsign, int qcopy, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap qmap) {
    using Cfg = ChunkCfg<C, D>;
    using T = typename CacheT<C>::Q;
    constexpr int NQ = Cfg::NQ, SB = Cfg::SB, BN = Cfg::BN, NS = Cfg::NS, KU = Cfg::KU, VR = Cfg::VR;
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
    // tile n of a row tile uses score buffer n % SB, and its value product that one's barrier.  Before
    // anyone waits for product n, product n - SB was waited for (for P's place, or by the scores that
    // took its buffer), so the barrier is at most one phase away and the parity is unambiguous
    auto pv_done = [&](int q, int b) { return bars + 8u * (2 * NS + NQ + 2 * NQ * SB + q * SB + b); };
    auto p_half = [&](int q, int b) { return bars + 8u * (2 * NS + NQ + 3 * NQ * SB + q * SB + b); };
    auto s_empty = [&](int q) { return bars + 8u * (2 * NS + NQ + 4 * NQ * SB + q); };
    // Codes of unit u arrive in area u % NRAW on barrier u % NRAWBAR, phase u / NRAWBAR.  With two converting
    // warpgroups the units of an area go to them in turn; a barrier per area alone would let one of them
    // wait for a phase while the one before, which only the other waited for, is still open, and take
    // its parity for the answer.  So a barrier's units are all one warpgroup's, which waits for every phase.
    // A full barrier says more: unit u was copied after unit u - NRAW had been converted, into a slot whose
    // earlier tile had been used, so the converters' waits on kv_empty are one phase away at most too (NS = NRAW there)
    static_assert(Cfg::NCONV <= 1 || Cfg::NS == Cfg::NRAW, "phases of kv_empty");
    auto raw_full = [&](int s) { return bars + 8u * (Cfg::NBAR - 1 - Cfg::NRAW - Cfg::NRAWBAR + s); };
    auto raw_empty = [&](int s) { return bars + 8u * (Cfg::NBAR - 1 - Cfg::NRAW + s); };
    const uint32_t raw_codes = base + Cfg::RAW_AT, raw_steps = raw_codes + Cfg::NRAW * Cfg::CODES;
    const uint32_t v_raw = bars + 8u * (Cfg::NBAR - 1), taddr_slot = bars + 8u * Cfg::NBAR, turn = taddr_slot + 4;

    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(kv_full(s), Cfg::Q8 ? 128 : 1);
            mbar_init(kv_empty(s), NQ);
        }
        mbar_init(v_raw, 1);
        for (int s = 0; s < Cfg::NRAWBAR; ++s) mbar_init(raw_full(s), 1);
        for (int s = 0; s < Cfg::NRAW; ++s) mbar_init(raw_empty(s), 128);
        for (int q = 0; q < NQ; ++q) {
            mbar_init(q_full(q), qcopy ? 1 : 128);
            mbar_init(s_empty(q), 128);
            for (int b = 0; b < SB; ++b) {
                mbar_init(pv_done(q, b), 1);
                mbar_init(s_full(q, b), 1);
                mbar_init(p_half(q, b), 128);
                mbar_init(p_full(q, b), 128);
            }
        }
        fence_mbar_init();
        asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(turn), "r"(0u) : "memory");
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
    const Ranges rg(total, ctas);
    const int64_t w0 = (int)blockIdx.x < ctas ? rg.start(blockIdx.x) : 0;
    const int64_t w1 = (int)blockIdx.x < ctas ? rg.start(blockIdx.x + 1) : 0;
    ChunkWalk k{};
    const int dealt = *plan.dealt ? *plan.nrt * a.Hk : 0;
    if (dealt) {
        chunk_deal(k, plan, a.Hk, dealt);
    } else if (w1 > w0) {
        k = chunk_find(plan, *plan.nrt, w0);
        k.left = w1 - w0;
        if (k.end() <= k.blk()) k.left = 0;  // the range ends before the item's first slot tile
    }
    uint32_t units = 0;  // key and value tiles so far: tile u sits in slot u % NS

    if (warp < 4 * NQ) {
        // ------------------------------------------------------------ a row per thread
        if constexpr (Cfg::ROW_REGS > 0) set_max_regs<true, Cfg::ROW_REGS>();
        const int q = warp >> 2, r = tid & 127, wr = r & ~31;  // wr: first row of the warp
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t ocol = lanes + Cfg::O_COL + q * D;
        const uint32_t qtile = base + q * Cfg::QB;
        const uint32_t mG = (uint32_t)((0x100000000ull + a.G - 1) / a.G);
        constexpr int CPR = D / 8;  // 16-byte chunks of a row
        // Queries come as tiled copies where the G heads of whole tokens make 128 rows, else (and with a
        // negative scale) as 16-byte copies of each warp's rows; either way into the products' operand layout
        // and while the item before is finished
        auto query_at = [&](int x) {
            const int row = wr + x / CPR, ch = x % CPR;
            return qtile + (ch >> 3) * (128 * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
        };
        auto fetch_q = [&](const ChunkWalk &w) {
            const int nrows = w.t.n * a.G, row0 = w.t.row0 + 128 * q;
            if (row0 >= nrows) return;
            if (!qcopy) {
#pragma unroll 1
                for (int i = 0; i < CPR; ++i) {
                    // rows past the last are any rows: nothing of them is written
                    const int x = i * 32 + lane, rr = min(row0 + wr + x / CPR, nrows - 1);
                    int g;
                    const int t = fast_div(rr, a.G, mG, g);
                    cp_async16(query_at(x), static_cast<const T *>(a.q) + (int64_t)(w.t.first + t) * a.ldq + (int64_t)(w.h * a.G + g) * a.hdq +
                                                8 * (x % CPR));
                }
            } else if (r == 0) {
                mbar_arrive_expect_tx(q_full(q), Cfg::QB);
#pragma unroll
                for (int p = 0; p < Cfg::NP; ++p)
                    tma_load_4d(qtile + p * (128 * 128), &qmap, 64 * p, 0, w.h, w.t.first + row0 / a.G, q_full(q));
            }
        };
        auto finish_q = [&]() {  // the thread's own 16-byte copies
            cp_async_wait();
            if (qsign) {
#pragma unroll 1
                for (int i = 0; i < CPR; ++i) {
                    const uint32_t at = query_at(i * 32 + lane);
                    const uint4 v = lds128(at);
                    sts128(at, v.x ^ qsign, v.y ^ qsign, v.z ^ qsign, v.w ^ qsign);
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(q_full(q));
        };
        if (tid == 0) a.desc[blockIdx.x].parts = 0;
        uint32_t done = 0;  // slot tiles of this row tile so far
        if (k.left > 0) fetch_q(k);
        while (k.left > 0) {
            const int blk0 = k.blk(), end = k.end();
            const int nrows = k.t.n * a.G, row0 = k.t.row0 + 128 * q;
            ChunkWalk nk = k;
            chunk_next(nk, plan, a.Hk, dealt);
            if (row0 < nrows) {
                if (!qcopy) finish_q();
                const int rr = row0 + r, pos0 = k.t.len - k.t.n;
                int g;
                const int pos = pos0 + fast_div(rr, a.G, mG, g);
                const int hi = rr < nrows ? pos : -1, lo = seen_from(pos, a.window);
                const int hi_min = pos0 + row0 / a.G;  // every row sees up to here, and from lo_max on
                const int lo_max = seen_from(pos0 + (min(row0 + 128, nrows) - 1) / a.G, a.window);
                float m = -INFINITY, l = 0.0f;
                for (int j = blk0; j < end; ++j, ++done) {
                    const int buf = SB == 1 ? 0 : (int)(done & 1);
                    const uint32_t scol = lanes + (Cfg::S_TURNS ? 0 : (q * SB + buf) * BN);
                    const int key0 = (k.t.kb0 + j) * BN;
                    const int c_hi = hi - key0, c_lo = lo - key0;  // visible columns
                    const bool edge = key0 + BN - 1 > hi_min || key0 < lo_max;
                    mbar_wait(s_full(q, buf), (done / SB) & 1);
                    tc_fence_after();
                    uint32_t s[Cfg::HOLD ? BN / 32 : 1][32];
                    auto mask = [&](uint32_t (&v)[32], int c0) {
                        if (edge) {
                            const int up = c_hi - c0, down = c_lo - c0;  // visible: down .. up
                            const uint32_t see = (up < 0 ? 0u : 0xffffffffu >> (31 - min(up, 31))) & (down > 31 ? 0u : 0xffffffffu << max(down, 0));
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!(see >> i & 1u)) v[i] = 0xff800000u;  // -inf
                        }
                    };
                    auto top = [&](const uint32_t (&v)[32]) {
                        float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int i = 0; i < 32; i += 2)
                            x[(i / 2) & 3] = fmaxf(fmaxf(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), x[(i / 2) & 3]);
                        return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
                    };
                    float mx = -INFINITY;
                    if constexpr (Cfg::HOLD) {
#pragma unroll
                        for (int c = 0; c < BN / 32; ++c) tmem_ld32(scol + 32 * c, s[c]);
                        tmem_wait_ld(s[0]);
#pragma unroll
                        for (int c = 1; c < BN / 32; ++c) tmem_loaded(s[c]);
                        tc_fence_before();
                        mbar_arrive(s_empty(q));  // P has columns of its own here
#pragma unroll
                        for (int c = 0; c < BN / 32; ++c) {
                            mask(s[c], 32 * c);
                            mx = fmaxf(mx, top(s[c]));
                        }
                    } else {
#pragma unroll 1
                        for (int c = 0; c < BN / 32; ++c) {
                            tmem_ld32(scol + 32 * c, s[0]);
                            tmem_wait_ld(s[0]);
                            mask(s[0], 32 * c);
                            mx = fmaxf(mx, top(s[0]));
                        }
                    }
                    if (!Cfg::P_OVER && done > 0) {  // P's place is free again
                        mbar_wait(pv_done(q, 0), (done - 1) & 1);
                        tc_fence_after();
                    }
                    // ---- rescale where some row of the warp needs it (the first tile starts O afresh)
                    if (j == blk0) {
                        m = mx;
                    } else {
                        const bool grown = (mx - m) * a.scale2 > 8.0f || (m == -INFINITY && mx > m);
                        if (__any_sync(0xffffffffu, grown)) {
                            const float mn = fmaxf(m, mx), f = mn > m ? exp2_approx((m - mn) * a.scale2) : 1.0f;
                            m = mn;
                            l *= f;
                            if (Cfg::P_OVER) {
                                mbar_wait(pv_done(q, (done - 1) % SB), ((done - 1) / SB) & 1);
                                tc_fence_after();
                            }
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) {
                                uint32_t o[16];
                                tmem_ld16(ocol + c, o);
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                tmem_st16(ocol + c, o);
                            }
                            tmem_wait_st();
                        }
                    }
                    // exponents x = S * sc - mz
                    const bool far = chunk_far(m, a.scale2);
                    const float sc = far ? a.scale_p2 : a.scale2;
                    const float mz = m == -INFINITY ? -Cfg::P_SHIFT : far ? m * sc : m * sc - Cfg::P_SHIFT;
                    // ---- P: chunk c of 32 scores becomes columns (words of a row) 16 c .. 16 c + 15
                    const uint64_t sc2 = pack_f32x2(sc, sc), mz2 = pack_f32x2(-mz, -mz);
                    uint64_t sum[2] = {0ull, 0ull};
#pragma unroll (Cfg::HOLD ? BN / 32 : 1)
                    for (int c = 0; c < BN / 32; ++c) {
                        uint32_t(&v)[32] = s[Cfg::HOLD ? c : 0];
                        if constexpr (!Cfg::HOLD) {
                            tmem_ld32(scol + 32 * c, v);
                            tmem_wait_ld(v);
                            if (!Cfg::P_OVER && c + 1 == BN / 32) {
                                tc_fence_before();
                                mbar_arrive(s_empty(q));
                            }
                            mask(v, 32 * c);
                        }
                        uint32_t p[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const uint64_t x = fma_f32x2(pack_b32x2(v[2 * i], v[2 * i + 1]), sc2, mz2);
                            float x0, x1;
                            unpack_f32x2(x, x0, x1);
                            x0 = exp2_approx(x0);
                            x1 = exp2_approx(x1);
                            sum[i & 1] = add_f32x2(sum[i & 1], pack_f32x2(x0, x1));
                            p[i] = pack2<T>(x0, x1);
                        }
                        tmem_st16((Cfg::P_OVER ? scol : lanes + Cfg::P_COL + q * (BN / 2)) + 16 * c, p);
                        if (c == BN / 64 - 1) {
                            tmem_wait_st();
                            tc_fence_before();
                            mbar_arrive(p_half(q, buf));
                        }
                    }
                    float l0, l1, l2, l3;
                    unpack_f32x2(sum[0], l0, l1);
                    unpack_f32x2(sum[1], l2, l3);
                    l += (l0 + l1) + (l2 + l3);
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(p_full(q, buf));
                }
                if (nk.left > 0) fetch_q(nk);  // no product reads this item's queries any more
                // ---- result
                mbar_wait(pv_done(q, (done - 1) % SB), ((done - 1) / SB) & 1);
                tc_fence_after();
                const bool whole = blk0 == 0 && end == k.t.nt;
                if (warp == 0 && blk0 == 0 && !whole) {
                    const int64_t s0 = w1 - k.left - k.u;  // the item's first unit
                    const int parts = rg.parts(blockIdx.x, s0 + k.t.nt + CHUNK_OV);
                    if (lane == 0) a.desc[blockIdx.x] = JoinDesc{parts, k.t.first, k.h, k.t.row0, k.t.n * a.G, {}};
                }
                const float inv = l > 0.0f ? 1.0f / l : l;  // nothing visible: 0
                const float top = m == -INFINITY ? 0.0f : m * a.scale2;
                const float ls = l > 0.0f ? top + (log2_approx(l) - (chunk_far(m, a.scale2) && m != -INFINITY ? 0.0f : Cfg::P_SHIFT))
                                          : l == 0.0f ? -INFINITY : l;
                float *part = a.part + (size_t)(2 * blockIdx.x + (blk0 == 0 ? 1 : 0)) * attn_part_floats(Cfg::ROWS, D);
                if (rr < nrows) {
                    if (!whole)
                        part[(size_t)Cfg::ROWS * D + 128 * q + r] = ls;
                    else if (a.lse)
                        a.lse[(int64_t)(k.t.first + pos - pos0) * a.Hq + k.h * a.G + g] = ls * LN2;
                }
                const int mine = rr < nrows ? (k.t.first + pos - pos0) * a.Hq + k.h * a.G + g : -1;  // the thread's row of out
                if (!whole) {
                    // columns in groups of 4, rows within: a warp's store is 512 contiguous bytes
                    float4 *dst = reinterpret_cast<float4 *>(part) + 128 * q + r;
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tmem_ld32(ocol + c, o);
                        tmem_wait_ld(o);
                        if (mine >= 0) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                dst[(c / 4 + i) * Cfg::ROWS] = make_float4(__uint_as_float(o[4 * i]) * inv, __uint_as_float(o[4 * i + 1]) * inv,
                                                                           __uint_as_float(o[4 * i + 2]) * inv, __uint_as_float(o[4 * i + 3]) * inv);
                        }
                    }
                } else {
                    // 64 bytes of each row at a time through the warp's own shared memory, so that a store
                    // writes whole sectors of 8 rows
                    const uint32_t st = base + Cfg::OUT_AT + warp * 2048;
                    auto place = [&](int row, int ch) { return st + row * 64 + ((ch ^ ((row >> 1) & 3)) << 4); };
                    auto flush = [&](int at, int pitch) {  // bytes `at` .. of rows of `pitch` bytes
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int row = 8 * i + lane / 4, orow = __shfl_sync(0xffffffffu, mine, row);
                            const uint4 v = lds128(place(row, lane & 3));
                            if (orow >= 0) *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(a.out) + (int64_t)orow * pitch + at + 16 * (lane & 3)) = v;
                        }
                        __syncwarp();
                    };
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tmem_ld32(ocol + c, o);
                        tmem_wait_ld(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
                        if (a.out_f32) {
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    sts128(place(lane, i), o[16 * x + 4 * i], o[16 * x + 4 * i + 1], o[16 * x + 4 * i + 2], o[16 * x + 4 * i + 3]);
                                flush((c + 16 * x) * 4, D * 4);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                auto two = [&](int e) { return pack2<T>(__uint_as_float(o[8 * i + e]), __uint_as_float(o[8 * i + e + 1])); };
                                sts128(place(lane, i), two(0), two(2), two(4), two(6));
                            }
                            flush(c * 2, D * 2);
                        }
                    }
                }
                tc_fence_before();  // the next item's products overwrite O once its P arrives
            } else if (nk.left > 0) {
                fetch_q(nk);
            }
            k = nk;
        }
    } else if (warp < Cfg::CONV_WARP) {
        if constexpr (Cfg::ISSUE_REGS > 0) set_max_regs<false, Cfg::ISSUE_REGS>();
        if (warp < Cfg::MMA_WARP + NQ) {
        // ------------------------------------------------------------ products: a warp per row tile
        constexpr uint32_t id_s = umma_idesc_16(128, BN, BF, false), id_o = umma_idesc_16(128, D, BF, true);
        constexpr uint32_t desc_hi = (uint32_t)(umma_desc_kmajor_sw128(0) >> 32);
        static_assert(desc_hi == (uint32_t)(umma_desc_mnmajor_sw128(0, VR * 128) >> 32), "one upper word");
        const uint32_t leader = lane == 0;
        const int q = NQ == 1 ? 0 : (int)warp_uniform((uint32_t)(warp - Cfg::MMA_WARP));
        const uint32_t s_col = warp_uniform(tmem + (Cfg::S_TURNS ? 0 : q * SB * BN)), o_col = warp_uniform(tmem + Cfg::O_COL + q * D);
        const uint32_t p_col = warp_uniform(Cfg::P_OVER ? tmem + q * SB * BN : tmem + Cfg::P_COL + q * (BN / 2));
        const uint32_t q_desc = warp_uniform((uint32_t)umma_desc_kmajor_sw128(base + q * Cfg::QB));
        uint32_t items = 0, n = 0;  // items; slot tiles of this row tile before the segment
        uint32_t other = 0;         // slot tiles of the other row tile before the segment (they take turns)
        bool both_before = false;   // the segment before had rows in both tiles
        uint32_t seg = 0;           // segments begun
        auto wait_turn = [&](uint32_t s) {  // until row tile 0 has begun segment s; bounded as every wait
            const unsigned long long t0 = globaltimer_ns();
            for (uint32_t spin = 1;; ++spin) {
                uint32_t v;
                asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(turn) : "memory");
                if (__any_sync(0xffffffffu, v >= s)) break;
                if ((spin & 255u) == 0 && __any_sync(0xffffffffu, globaltimer_ns() - t0 > WAIT_NS)) {
                    if (lane == 0) atomicOr(&g_qg_dev_err, DEVERR_TIMEOUT);
                    break;
                }
            }
        };
        // S = Q K^T of slot tile j of the segment, whose keys are units u ..
        auto scores = [&](int j, bool both, uint32_t u) {
            const uint32_t t = n + j, buf = t % SB;
            // the buffer's last scores have been read, and P that took their place
            if constexpr (Cfg::S_TURNS) {
                if (q == 1) {
                    // Row tile 0 takes segments that have no rows in this tile alone.  Its barrier's parity says
                    // nothing until it has come to this segment, which it publishes
                    if (j == 0) wait_turn(seg);
                    mbar_wait(s_empty(0), (other + j) & 1);
                } else {
                    if (j > 0 ? both : both_before)
                        mbar_wait(s_empty(1), (other + j - 1) & 1);
                    else if (t > 0)
                        mbar_wait(s_empty(0), (t - 1) & 1);
                    if (j == 0 && lane == 0) asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(turn), "r"(seg) : "memory");
                }
            } else if (t >= SB) {
                if (Cfg::P_OVER)
                    mbar_wait(pv_done(q, buf), (t / SB - 1) & 1);
                else
                    mbar_wait(s_empty(q), (t - 1) & 1);
            }
            const uint32_t dst = warp_uniform(s_col + buf * BN);
#pragma unroll
            for (int h = 0; h < KU; ++h, ++u) {
                const uint32_t slot = u % NS;
                mbar_wait(kv_full(slot), (u / NS) & 1);
                tc_fence_after();
                const uint32_t kd = warp_uniform((uint32_t)umma_desc_kmajor_sw128(kv0 + slot * Cfg::TILE));
                const uint32_t qd = q_desc + h * Cfg::PKU * (128 * 128 / 16);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4 * Cfg::PKU; ++i)
                    umma_f16_w(leader, dst, qd + (i / 4) * (128 * 128 / 16) + 2 * (i % 4), kd + (i / 4) * (BN * 128 / 16) + 2 * (i % 4),
                               desc_hi, id_s, (h | i) != 0);
                if (h == KU - 1) umma_commit_w(leader, s_full(q, buf));
                umma_commit_w(leader, kv_empty(slot));
            }
        };
        // O (+)= P V over a half of slot tile t, whose values are units u ..
        auto product = [&](uint32_t t, bool fresh, uint32_t u, auto which) {
            constexpr int half = decltype(which)::value;
            const uint32_t buf = t % SB, src = warp_uniform(p_col + (Cfg::P_OVER ? buf * BN : 0));
            const uint32_t slot = (KU == 2 ? u + half : u) % NS, phase = ((KU == 2 ? u + half : u) / NS) & 1;
            mbar_wait(kv_full(slot), phase);
            const uint32_t vd = warp_uniform((uint32_t)umma_desc_mnmajor_sw128(kv0 + slot * Cfg::TILE, VR * 128));
            mbar_wait(half ? p_full(q, buf) : p_half(q, buf), (t / SB) & 1);
            tc_fence_after();
            __syncwarp();
#pragma unroll
            for (int i = 0; i < BN / 32; ++i) {
                const int p = half * (BN / 32) + i;  // 16 slots of P
                umma_f16_ta_w(leader, o_col, src + 8 * p, vd + (KU == 2 ? i : p) * (2048 / 16), desc_hi, id_o, p ? 1u : !fresh);
            }
            if (half) umma_commit_w(leader, pv_done(q, buf));
            if (half || KU == 2) umma_commit_w(leader, kv_empty(slot));
        };
        using First = std::integral_constant<int, 0>;
        using Second = std::integral_constant<int, 1>;
        while (k.left > 0) {
            const int taken = k.end() - k.blk();
            ++seg;
            if (q == 0 || k.t.row0 + 128 < k.t.n * a.G) {
                mbar_wait(q_full(q), items & 1);
                ++items;
                const bool both = NQ == 2 && k.t.row0 + 128 < k.t.n * a.G;
                for (int j = 0; j <= taken; ++j) {  // the values of a tile come after the next one's keys
                    if (j < taken) {
                        scores(j, both, units);
                        units += KU;
                    }
                    if (j > 0) {
                        product(n + j - 1, j == 1, units, First{});
                        product(n + j - 1, j == 1, units, Second{});
                        units += KU;
                    }
                }
                n += taken;
                both_before = both;
                if (both || q == 1) other += taken;
            } else {  // no rows in this tile: its share of every unit's release
                other += taken;
                for (int j = 0; j < 2 * KU * taken; ++j, ++units) {
                    mbar_wait(kv_full(units % NS), (units / NS) & 1);
                    if (lane == 0) mbar_arrive(kv_empty(units % NS));
                }
            }
            chunk_next(k, plan, a.Hk, dealt);
        }
        // complete already on the normal path; after a wait gave up, let products in flight end
        if (lane == 0 && n) mbar_drain(pv_done(q, (n - 1) % SB), ((n - 1) / SB) & 1, DRAIN_NS);
        __syncwarp();
        } else if (warp == Cfg::MMA_WARP + NQ) {
        // ------------------------------------------------------------ copies
        // A unit is one box per page part and panel, each issued by a lane of its own.  Lane b looks up the
        // page of the tile's slots 16 b .. one tile ahead.
        struct Place {
            int page, slot;
        };
        auto lookup = [&](const ChunkWalk &w, int j) {
            Place p{a.bt.n_pages, 0};  // out of range: zeros
            const int key = (w.t.kb0 + j) * BN + 16 * lane;
            if (w.left > 0 && lane < BN / 16 && key < w.t.len) {
                p.page = a.bt.pages[w.t.b * a.bt.table_stride + key / a.bt.page];
                p.slot = key % a.bt.page;
            }
            return p;
        };
        uint32_t raws = 0;
        // Unit h of the keys or values of a tile; a lane's box and panel, and the 16 slots whose steps it copies
        auto copy = [&](const Place &p, int h, int head, bool val, int tile) {
            constexpr int KP = Cfg::Q8 ? Cfg::KCP : Cfg::PKU, VP = Cfg::Q8 ? Cfg::VCP : Cfg::NP;
            const int rows = val ? VR : BN, first = val ? h * VR : 0;
            const int box = val ? lane / VP : lane / KP, panel = val ? lane % VP : lane % KP;
            const int from = first + box * box_rows;  // the box's first slot in the tile
            int page = __shfl_sync(0xffffffffu, p.page, (from / 16) & 31);
            const int s0 = __shfl_sync(0xffffffffu, p.slot, (from / 16) & 31);
            if ((unsigned)page >= (unsigned)a.bt.n_pages) page = a.bt.n_pages;
            if constexpr (Cfg::Q8) {
                // codes and steps as they are, for the converting warpgroups
                const uint32_t slot = units % Cfg::NRAW, bar = raw_full(units % Cfg::NRAWBAR);
                const bool here = box * box_rows < rows, steps = here && panel == 0, good = steps && page < a.bt.n_pages;
                const uint32_t BS = box_rows * (D / 32) * 2;  // bytes of a box's steps
                const uint32_t sdst = raw_steps + slot * Cfg::STEPS + box * BS;
                if (units >= Cfg::NRAW) mbar_wait(raw_empty(slot), (units / Cfg::NRAW - 1) & 1);
                if (steps && !good) {
                    for (uint32_t x = 0; x < BS; x += 16) sts128(sdst + x, 0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();  // a later bulk copy writes the same place
                }
                const uint32_t goods = __popc(__ballot_sync(0xffffffffu, good));
                __syncwarp();  // the zeros are written before the arrival below
                if (lane == 0) mbar_arrive_expect_tx(bar, Cfg::CODES + goods * BS);
                __syncwarp();
                if (here)
                    tma_load_4d(raw_codes + slot * Cfg::CODES + panel * (rows * Cfg::CPANEL) + box * box_rows * Cfg::CPANEL, val ? &vmap : &kmap,
                                Cfg::CPANEL * ((val ? 0 : h) + panel), s0, head, page, bar);
                if (good)
                    bulk_g2s(sdst, (val ? a.vd : a.kd) + page * a.step_stride + ((int64_t)head * a.bt.page + s0) * (D / 32), BS, bar);
            } else {
                const uint32_t slot = units % NS;
                // Slots that no row sees may hold anything, and 0 * NaN is not 0: their values become zeros before
                // the unit counts as full
                int z0 = 0, z1 = VR;
                if (val) {
                    const int key0 = (k.t.kb0 + tile) * BN + h * VR;
                    const int seen_lo = seen_from(k.t.len - k.t.n + k.t.row0 / a.G, a.window);
                    z0 = min(VR, max(0, seen_lo - key0)), z1 = min(VR, max(0, k.t.len - key0));
                }
                const bool mend = z0 > 0 || z1 < VR;
                const uint32_t bar = mend ? v_raw : kv_full(slot);
                if (units >= NS) mbar_wait(kv_empty(slot), (units / NS - 1) & 1);
                if (lane == 0) mbar_arrive_expect_tx(bar, Cfg::TILE);
                __syncwarp();
                if (box * box_rows < rows)
                    tma_load_4d(kv0 + slot * Cfg::TILE + panel * (rows * 128) + box * box_rows * 128, val ? &vmap : &kmap,
                                64 * ((val ? 0 : h * Cfg::PKU) + panel), s0, head, page, bar);
                if (mend) {
                    mbar_wait(v_raw, raws++ & 1);
                    for (int x = lane; x < (z0 + VR - z1) * (D / 8); x += 32) {
                        const int row = x / (D / 8), ch = x % (D / 8);
                        sts128(kv0 + slot * Cfg::TILE + (ch >> 3) * (VR * 128) + (row < z0 ? row : row - z0 + z1) * 128 + (ch & 7) * 16, 0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(kv_full(slot));
                }
            }
            ++units;
        };
        ChunkWalk nx = k;  // the tile whose pages are looked up
        int nj = k.blk();
        auto ahead = [&]() {
            if (nx.left > 0 && ++nj >= nx.end()) {
                chunk_next(nx, plan, a.Hk, dealt);
                nj = nx.blk();
            }
            return lookup(nx, nj);
        };
        Place prev{}, cur = lookup(nx, nj), next = ahead();
        while (k.left > 0) {
            const int blk0 = k.blk(), end = k.end();
            // the values of a tile come after the next one's keys; one place for all copies keeps the code short
#pragma unroll 1
            for (int j = blk0; j <= end; ++j) {
#pragma unroll 1
                for (int x = j < end ? 0 : KU; x < (j > blk0 ? 2 * KU : KU); ++x) {
                    const bool val = x >= KU;
                    copy(Place{val ? prev.page : cur.page, val ? prev.slot : cur.slot}, val ? x - KU : x, k.h, val, j - 1);
                }
                if (j < end) {
                    prev = cur;
                    cur = next;
                    next = ahead();
                }
            }
            chunk_next(k, plan, a.Hk, dealt);
        }
        if (lane == 0) {  // complete already on the normal path
            if constexpr (Cfg::Q8) {
                for (uint32_t s = 0; s < Cfg::NRAWBAR && s < units; ++s)
                    mbar_drain(raw_full(s), ((units - 1 - s) / Cfg::NRAWBAR) & 1, DRAIN_NS);
            } else {
                for (uint32_t s = 0; s < NS && s < units; ++s) mbar_drain(kv_full(s), ((units - 1 - s) / NS) & 1, DRAIN_NS);
            }
        }
        __syncwarp();
        }
    } else if constexpr (Cfg::Q8) {
        // ------------------------------------------------------------ 8-bit codes to fp16 tiles
        // Thread ct converts every 128th 16-code chunk of its warpgroup's units.
        set_max_regs<Cfg::CONV_REGS >= Cfg::LAUNCH_REGS, Cfg::CONV_REGS>();
        const int cw = (warp - Cfg::CONV_WARP) / 4, ct = (tid - Cfg::CONV_WARP * 32) & 127;
        constexpr int PER = Cfg::CODES / 16 / 128;  // chunks per thread
        int kt = k.blk(), vt = -1, blk0 = kt, end = k.end();  // the last key and value tiles begun
        int h = -1;
        bool val = false, on = k.left > 0;
        auto next_unit = [&]() {  // the order of the copies
            if (++h < KU) return;
            h = 0;
            if (!val) {
                if (kt == blk0 && kt + 1 < end) {
                    ++kt;
                } else {
                    val = true;
                    vt = max(blk0, kt - 1);
                }
            } else if (kt + 1 < end) {
                val = false;
                ++kt;
            } else if (vt < kt) {
                ++vt;
            } else {
                chunk_next(k, plan, a.Hk, dealt);
                val = false;
                on = k.left > 0;
                blk0 = kt = k.blk();
                end = k.end();
            }
        };
        auto convert = [&](uint32_t n, auto is_val) {  // unit number n
            constexpr bool VAL = decltype(is_val)::value;
            constexpr int ROWSU = VAL ? VR : BN, CPR = Cfg::CODES / 16 / ROWSU, RPS = 128 / CPR;  // rows, chunks of a row, rows of a step of i
            constexpr int CC = Cfg::CPANEL / 16;                                                  // chunks of a panel's row
            const uint32_t raw = n % Cfg::NRAW, slot = n % NS;
            // Eight lanes at a time read codes and write tiles without bank conflicts: four chunks of one row and
            // the four of the other half of the next (both rows' panels meet at one bank otherwise)
            const int odd = (ct >> 2) & 1;
            const int r0 = CPR == 4 ? ct / 4 : 2 * (ct / (2 * CPR)) + odd;
            const int ch = CPR == 4 ? ct % 4 : (CPR == 16 ? (ct >> 4 & 1) * 8 : 0) + 4 * (odd ^ (ct >> 3 & 1)) + (ct & 3);
            mbar_wait(raw_full(n % Cfg::NRAWBAR), (n / Cfg::NRAWBAR) & 1);
            // slots that no row sees may hold anything: they become zeros
            const int key0 = (k.t.kb0 + (VAL ? vt : kt)) * BN + (VAL ? h * VR : 0);
            const int seen_lo = seen_from(k.t.len - k.t.n + k.t.row0 / a.G, a.window);
            const int from = max(0, seen_lo - key0), to = k.t.len - key0;  // rows of slots
            if (n >= NS) mbar_wait(kv_empty(slot), (n / NS - 1) & 1);
            // a short loop: the roles run at once and share the instruction cache (512 tokens after 8000, dim 256:
            // 146 us as it is or unrolled twice, 149 four times)
#pragma unroll 1
            for (int i = 0; i < PER; ++i) {
                const int row = i * RPS + r0;
                const uint4 c = lds128(raw_codes + raw * Cfg::CODES + (ch / CC) * (ROWSU * Cfg::CPANEL) + row * Cfg::CPANEL +
                                       (((ch % CC) ^ (Cfg::CPANEL == 128 ? row & 7 : (row >> 1) & 3)) << 4));
                const uint32_t d = lds16(raw_steps + raw * Cfg::STEPS + (row * (D / 32) + (VAL ? 0 : h * (Cfg::PKU * 2)) + ch / 2) * 2);
                const uint32_t dd = row >= from && row < to ? d | d << 16 : 0u;
                const uint32_t in[4] = {c.x, c.y, c.z, c.w};
                uint32_t x[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t b = in[e] ^ 0x80808080u;
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t f = codes_to_f16(b, y ? 0x4342 : 0x4140);
                        const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&f), *reinterpret_cast<const __half2 *>(&dd));
                        x[2 * e + y] = *reinterpret_cast<const uint32_t *>(&r);
                    }
                }
                const uint32_t row_at = kv0 + slot * Cfg::TILE + (ch >> 2) * (ROWSU * 128) + row * 128;
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    sts128(row_at + (((2 * (ch & 3) + y) ^ (row & 7)) << 4), x[4 * y], x[4 * y + 1], x[4 * y + 2], x[4 * y + 3]);
            }
            // the copies that come next write the codes' place, and the products read the tile, by the async proxy
            fence_proxy_async_smem();
            mbar_arrive(raw_empty(raw));
            mbar_arrive(kv_full(slot));
        };
        next_unit();
        for (uint32_t n = 0; on; ++n, next_unit()) {
            if ((int)(n % Cfg::NCONV) != cw) continue;
            if (val)
                convert(n, std::true_type{});
            else
                convert(n, std::false_type{});
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == Cfg::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, Cfg::COLS);
    }
}

// Merges the partial results of the items that range boundaries cut and clears the rows of no sequence: as
// attn_join_kernel, block (x, y) for the item that CTA x described, its y-th share.  Rows past the last hold nothing: theirs
// are read but not written.
template <class T, int D>
__global__ void __launch_bounds__(256) attn_chunk_join_kernel(const AttnArgs a) {
    constexpr int ROWS = ChunkCfg<CACHE_F16, D>::ROWS;
    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.x == gridDim.x - 1) {
        clear_outside<T>(a, D);
        return;
    }
    const JoinDesc jd = a.desc[blockIdx.x];
    const int parts = jd.parts, lane = threadIdx.x & 31;
    if (parts == 0) return;
    auto part = [&](int i) {  // the item ends the first range and starts the others
        return a.part + (size_t)(2 * ((int)blockIdx.x + i) + (i == 0 ? 1 : 0)) * attn_part_floats(ROWS, D);
    };
    // a warp takes a group of 4 columns of 32 rows, as they were written
    const int warp = threadIdx.x >> 5;
    constexpr int RG = ROWS / 32, CG = D / 4;  // row groups, column groups
    for (int x = blockIdx.y * 8 + warp; x < RG * CG; x += 8 * gridDim.y) {
        const int r = (x / CG) * 32 + lane, c = x % CG, rr = jd.row0 + r;
        if (jd.row0 + (x / CG) * 32 >= jd.nrows) break;
        float mx = -INFINITY;
        for (int i = 0; i < parts; ++i) mx = fmaxf(mx, part(i)[(size_t)ROWS * D + r]);
        const float mz = mx == -INFINITY ? 0.0f : mx;
        float sum = 0.0f, v[4] = {};
#pragma unroll 4
        for (int i = 0; i < parts; ++i) {
            const float *p = part(i);
            const float w = exp2_approx(p[(size_t)ROWS * D + r] - mz);
            const float4 o = reinterpret_cast<const float4 *>(p)[c * ROWS + r];
            sum += w;
            v[0] = fmaf(w, o.x, v[0]), v[1] = fmaf(w, o.y, v[1]), v[2] = fmaf(w, o.z, v[2]), v[3] = fmaf(w, o.w, v[3]);
        }
        const float inv = sum > 0.0f ? 1.0f / sum : sum;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] *= inv;
        if (rr < jd.nrows) {
            const int64_t row = (int64_t)(jd.first + rr / a.G) * a.Hq + jd.h * a.G + rr % a.G;
            if (a.out_f32)
                store_vec<float, 4>(static_cast<float *>(a.out) + row * D + 4 * c, v);
            else
                store_vec<T, 4>(static_cast<T *>(a.out) + row * D + 4 * c, v);
            if (a.lse && c == 0) a.lse[row] = sum > 0.0f ? (mz + log2_approx(sum)) * LN2 : sum == 0.0f ? -INFINITY : sum;
        }
    }
}

// ----------------------------------------------------------------------------- host
static int chunk_rows(int D) { return D == 256 ? 128 : 256; }

size_t attn_chunk_workspace(int D, int G, int tokens, int batch, int sms) {
    const int rows = chunk_rows(D);
    const size_t parts = (size_t)sms * 2 * attn_part_floats(rows, D) * sizeof(float);
    return parts + chunk_plan_bytes(chunk_max_tiles(rows, G, tokens, batch));
}

static int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

// Whether the current device gives the kernel what it needs.
template <int C, int D>
static bool chunk_ready() {
    using Cfg = ChunkCfg<C, D>;
    static std::mutex mu;
    static std::set<std::pair<const void *, int>> done;
    const void *kern = (const void *)attn_chunk_kernel<C, D>;
    return once_per_device(done, mu, kern, [&] {
        if (Cfg::WGS > 2) {  // the warpgroups trade registers out of exactly this allocation
            cudaFuncAttributes fa;
            if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess || fa.numRegs != Cfg::LAUNCH_REGS) return false;
        }
        return allow_smem(kern, Cfg::BYTES);
    });
}

template <int C, int D>
static int chunk_run(const AttnArgs &in, const qg_paged &c, int sms, cudaStream_t s) {
    using Cfg = ChunkCfg<C, D>;
    using T = typename CacheT<C>::Q;
    static_assert(Cfg::BYTES <= SMEM_MAX, "shared memory of the chunk kernel");
    AttnArgs a = in;
    const int64_t tiles = chunk_max_tiles(Cfg::ROWS, a.G, a.bt.tokens, a.bt.batch);
    const ChunkPlan plan = chunk_plan_at(reinterpret_cast<uint8_t *>(a.part + (size_t)sms * 2 * attn_part_floats(Cfg::ROWS, D)), tiles);
    // the maximum is taken over unscaled scores: a negative scale goes into the queries' signs, and
    // a scale of zero is a small one (masked scores stay -inf)
    const uint32_t qsign = a.scale2 < 0.0f ? 0x80008000u : 0u;
    a.scale2 = std::max(std::abs(a.scale2), 1e-30f);
    a.scale_p2 = std::exp2(std::floor(std::log2(a.scale2)));
    const int box = gcd(c.page, Cfg::VR);
    CUtensorMap km{}, vm{};
    const bool qcopy = 128 % a.G == 0 && !qsign;
    CUtensorMap qm{};
    if (qcopy && !attn_query_map(&qm, a, c.type == QG_BF16, D)) return QG_ECUDA;
    if (!attn_tensor_map(&km, c, c.k, box) || !attn_tensor_map(&vm, c, c.v, box)) return QG_ECUDA;
    if (!chunk_ready<C, D>()) return QG_ECUDA;
    if (!launch_programmatic(attn_plan_kernel, dim3(1), PLAN_THREADS, 0, s, a, plan, Cfg::ROWS, Cfg::BN, (int)tiles, sms)) return QG_ECUDA;
    auto kern = attn_chunk_kernel<C, D>;
    if (!launch_programmatic(kern, dim3((unsigned)sms), Cfg::THREADS, Cfg::BYTES, s, a, plan, box, qsign, (int)qcopy, km, vm, qm)) return QG_ECUDA;
    auto join = attn_chunk_join_kernel<T, D>;
    return launch_programmatic(join, dim3((unsigned)sms, 16), 256, 0, s, a) ? QG_OK : QG_ECUDA;
}

template <int C>
static int chunk_dim(const AttnArgs &a, const qg_paged &c, int sms, cudaStream_t s) {
    return c.dim == 64 ? chunk_run<C, 64>(a, c, sms, s) : c.dim == 128 ? chunk_run<C, 128>(a, c, sms, s) : chunk_run<C, 256>(a, c, sms, s);
}
int attn_chunk(const AttnArgs &a, const qg_paged &c, int sms, cudaStream_t s) {
    return c.type == QG_F16    ? chunk_dim<CACHE_F16>(a, c, sms, s)
           : c.type == QG_BF16 ? chunk_dim<CACHE_BF16>(a, c, sms, s)
                               : chunk_dim<CACHE_Q8>(a, c, sms, s);
}

int attn_chunk_dev_err_take(unsigned int *err) {
    unsigned int zero = 0;
    if (cudaMemcpyFromSymbol(err, g_qg_dev_err, sizeof(*err)) != cudaSuccess) return QG_ECUDA;
    if (cudaMemcpyToSymbol(g_qg_dev_err, &zero, sizeof(zero)) != cudaSuccess) return QG_ECUDA;
    return QG_OK;
}

}  // namespace qg
