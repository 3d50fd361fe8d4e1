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
};

// First slot that a row at position pos sees (window 0: all).  No difference that could pass 32 bits: a window
// of 2^31 - 1 over a sequence that begins with padding (pos < 0) is a call like any other.
__device__ __forceinline__ int seen_from(int pos, int window) { return window && pos >= window ? pos - window + 1 : 0; }

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

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
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

// The chunk kernel (qg_chunk.cu): many rows per sequence, and its workspace.
int attn_chunk(const AttnArgs &a, const qg_paged &c, int sms, cudaStream_t s);
size_t attn_chunk_workspace(int D, int G, int tokens, int batch, int sms);
int attn_chunk_dev_err_take(unsigned int *err);

}  // namespace qg
