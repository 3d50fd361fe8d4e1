// qg_attn.cuh -- what the two attention kernels share: arguments, tensor maps of the cache
// pools, the work list and the layout of partial results.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "qg_types.cuh"

namespace qg {

// What the join kernel merges: the item whose first slots a CTA took and whose end it left to others.
// Every CTA writes its own.
struct JoinDesc {
    int parts;        // partial results, in this CTA's range and the ones after (0: nothing to merge)
    int first, h;     // first token of the sequence, cache head
    int row0, nrows;  // first row of the tile, rows of the sequence
    int pad[3];
};

// What the kernels are compiled for (QG_MOD): causal or windowed attention; the same with other masks; with those and
// capped scores; and with those and a bias that falls with the distance, capped scores or not.  The row kernel is
// compiled for the first and for MOD_SHAPED, which does the rest there too.
enum { MOD_PLAIN, MOD_SHAPED, MOD_CAPPED, MOD_BIASED };

// What changes scores and masks (null: nothing), as the kernels read it.
struct Shape {
    float cap_in, cap_out;     // score = cap_out * tanh(cap_in * S), in powers of two (cap_out 0: not capped)
    float poly[5];             // chunk kernel: cap_out times the coefficients of tanh_near,
    float small[3];            // those of tanh_small, in S: score = S (small[0] + S^2 (small[1] + S^2 small[2])) up to
    float small_to;            // this |S| (below 0: nowhere)
    const float *slopes;       // Hq
    const int32_t *prefix;     // batch: the first slots, which every token of the sequence sees
    const int32_t *first;      // tokens: no slot before it is seen
    const uint32_t *tree;      // tokens x words: bit j: the sequence's new token j is seen
    int words;
    const int32_t *positions;  // tokens, beside a tree: positions where they are not the slots
};

struct AttnArgs {
    Batch bt;
    const void *q;
    int64_t ldq, hdq;  // elements between tokens, between heads
    void *out;         // tokens x Hq x D, contiguous
    float *lse;        // tokens x Hq, or NULL
    int Hq, Hk, G;     // G = Hq / Hk query heads share one cache head
    int out_f32;       // out is fp32 instead of the queries' type
    int window;        // 0: none
    float scale2;      // scale * log2(e): the kernels work in powers of two
    float scale_p2;    // the power of two below it (chunk kernel)
    const f16 *kd, *vd;
    int64_t step_stride;
    float *part;       // partial results (attn_part_floats each)
    JoinDesc *desc;    // one per CTA
    Shape sh;
};

// First slot that a row at position pos sees (window 0: all).  No difference that could pass 32 bits: a window
// of 2^31 - 1 over a sequence that begins with padding (pos < 0) is a call like any other.
__device__ __forceinline__ int seen_from(int pos, int window) { return window && pos >= window ? pos - window + 1 : 0; }

// The slots that new token i of sequence b sees: lo .. hi, and beside a tree those of its mask, which start at slot
// `base` of the sequence.  A token that sees nothing has hi = -1 and lo = INT_MAX.
struct Seen {
    int hi, lo, pos;
};
__device__ __forceinline__ Seen seen_by(const AttnArgs &a, const Seq &s, int b, int i) {
    const int slot = s.len - s.n + i, t = s.first + i;
    Seen r{-1, 0x7fffffff, slot};
    if (slot < 0) return r;  // padding
    if (a.sh.tree) {
        if (a.sh.positions) r.pos = a.sh.positions[t];
        r.hi = s.len - s.n - 1;
        r.lo = min(seen_from(r.pos, a.window), 0x7ffffffe);
    } else {
        r.hi = a.sh.prefix ? min(max(slot, max(a.sh.prefix[b], 0) - 1), s.len - 1) : slot;
        r.lo = seen_from(slot, a.window);
        if (a.sh.first) r.lo = max(r.lo, a.sh.first[t]);
        if (r.lo > r.hi) r.hi = -1, r.lo = 0x7fffffff;
    }
    return r;
}
// The first slot that the token needs, its own mask's included.
__device__ __forceinline__ int needs_from(const AttnArgs &a, const Seq &s, const Seen &v) {
    return a.sh.tree && v.lo != 0x7fffffff ? min(v.lo, max(s.len - s.n, 0)) : v.lo;
}
// How far positions are apart.  Whole numbers are subtracted, as fp32 does not hold positions past 2^24, and to one without
// a sign, as a caller's positions may be 2^32 apart.
__device__ __forceinline__ float distance(int p, int j) { return (float)__sad(p, j, 0u); }
// 32 bits of a row of a tree's mask from bit `at` on; the bits before 0 are set, those past the row are not.
__device__ __forceinline__ uint32_t tree_bits(const uint32_t *row, int words, int at) {
    const int w = at >> 5;
    const uint32_t lo = w < 0 ? 0xffffffffu : w < words ? row[w] : 0u, hi = w + 1 < 0 ? 0xffffffffu : w + 1 < words ? row[w + 1] : 0u;
    return __funnelshift_r(lo, hi, at & 31);
}

// tanh(x) for |x| <= TANH_NEAR: x times a polynomial in x^2 (our own fit to the least largest relative error: 7e-7 as
// evaluated).  Beyond it 1 - 2 / (1 + e^2x), which loses small x in the 1.
constexpr float TANH_NEAR = 0.75f;
constexpr float TANH_C0 = 0x1.ffffeep-1f, TANH_C1 = -0x1.554802p-2f, TANH_C2 = 0x1.0f8b42p-3f, TANH_C3 = -0x1.9a0facp-5f, TANH_C4 = 0x1.a7ad9ep-7f;
// And x (S0 + x^2 (S1 + x^2 S2)) for |x| <= TANH_SMALL: 5e-7.
constexpr float TANH_SMALL = 0.25f;
constexpr float TANH_S0 = 0x1.fffff2p-1f, TANH_S1 = -0x1.553762p-2f, TANH_S2 = 0x1.06ff0ap-3f;
__device__ __forceinline__ float tanh_near(float x) {
    const float u = x * x;
    return x * fmaf(u, fmaf(u, fmaf(u, fmaf(u, TANH_C4, TANH_C3), TANH_C2), TANH_C1), TANH_C0);
}

// One partial result: rows x D fp32 (normalised), then rows base-2 logarithms of the sums.
__host__ __device__ constexpr size_t attn_part_floats(int rows, int D) { return (size_t)rows * D + rows; }

// Work units cut into one range per CTA; range c starts at start(c).
struct Ranges {
    int64_t per;
    int rest, ctas;
    __device__ __forceinline__ Ranges(int64_t total, int n) : per(total / n), rest((int)(total % n)), ctas(n) {}
    __device__ __forceinline__ int64_t start(int c) const { return per * c + rest * c / ctas; }
    // Ranges that hold a part of the item that ends before unit s1, of which range c has the first; whole warp.
    __device__ __forceinline__ int parts(int c, int64_t s1) const {
        int n = 1;
        for (int i = c + 1; i < ctas; i += 32) {
            const int k = i + (threadIdx.x & 31);
            n += __popc(__ballot_sync(0xffffffffu, k < ctas && start(k) < s1));
        }
        return n;
    }
};

constexpr int DEC_ROWS = 16;  // rows of a tile of the row kernel at most

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float log2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// x / d and x % d for 0 <= x < 2^31 with m = ceil(2^32 / d).
__device__ __forceinline__ int fast_div(int x, int d, uint32_t m, int &rem) {
    int q = d == 1 ? x : (int)__umulhi((uint32_t)x, m);
    rem = x - q * d;
    if (rem < 0) {
        --q;
        rem += d;
    }
    return q;
}

__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}

// Tokens before the first sequence's and after the last one's see nothing: zeros, and -inf as the logarithm.  The last
// column of a join kernel's blocks writes them, so that the others' chain of loads is not longer for it (T: type
// of the queries).
template <class T>
__device__ __forceinline__ void clear_outside(const AttnArgs &a, int D) {
    const int lo = min(max(a.bt.q_start[0], 0), a.bt.tokens), hi = min(max(a.bt.q_start[a.bt.batch], 0), a.bt.tokens);
    for (int64_t i = blockIdx.y; i < (int64_t)lo + a.bt.tokens - hi; i += gridDim.y) {
        const int64_t row = (i < lo ? i : hi + i - lo) * a.Hq;
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(a.out) + row * D * (a.out_f32 ? 4 : sizeof(T)));
        const int chunks = a.Hq * (D / (a.out_f32 ? 4 : 8));
        for (int x = threadIdx.x; x < chunks; x += blockDim.x) dst[x] = make_uint4(0, 0, 0, 0);
        if (a.lse)
            for (int x = threadIdx.x; x < a.Hq; x += blockDim.x) a.lse[row + x] = -INFINITY;
    }
}

// 4-D tiled copy global -> shared: box at (element, slot, head, page); out-of-range pages give
// zeros.  The element coordinate is always a multiple of 128 bytes (64 where rows are 64).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int e, int slot, int head, int page,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(map), "r"(e), "r"(slot), "r"(head), "r"(page), "r"(bar)
        : "memory");
}

// Tensor map of one pool (keys or values): rows of `dim` elements, copied as boxes of `rows`
// slots x one swizzled panel (128 bytes of a row, or the whole row where it is 64 bytes).
// Host; false when the driver refuses.
bool attn_tensor_map(CUtensorMap *map, const qg_paged &c, const void *base, int rows);

// Tensor map of the queries for boxes of 128 rows x 128 bytes: the G heads of a cache head for
// 128 / G tokens, in that order (128 % G == 0).
bool attn_query_map(CUtensorMap *map, const AttnArgs &a, bool is_bf16, int D);

// Four int8 codes of a word as fp16 pairs (exact): code + 128 goes under the exponent of 1024.
__device__ __forceinline__ uint32_t codes_to_f16(uint32_t biased, uint32_t sel) {
    const uint32_t m = prmt(biased, 0x64646464u, sel);
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&m), __half2half2(__ushort_as_half(0x6480)));  // 1152
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ float tanh_any(float x) {
    const float r = rcp_approx(1.0f + exp2_approx(x * (2.0f * LOG2E)));
    return fabsf(x) <= TANH_NEAR ? tanh_near(x) : fmaf(-2.0f, r, 1.0f);
}

// The kernels by what they are compiled for: rows (qg_rows.cu): up to 8 nr rows of
// heads per sequence and cache head at a time; chunk (qg_chunk.cu): many, and its workspace.  _take: reads and clears the
// device error word.
template <int MOD>
int attn_rows(const AttnArgs &a, const qg_paged &c, int nr, int sms, cudaStream_t s);
template <int MOD>
int attn_chunk(const AttnArgs &a, const qg_paged &c, int sms, cudaStream_t s);
size_t attn_chunk_workspace(int D, int G, int tokens, int batch, int sms);
template <int MOD>
int attn_rows_dev_err_take(unsigned int *err);
template <int MOD>
int attn_chunk_dev_err_take(unsigned int *err);

}  // namespace qg
