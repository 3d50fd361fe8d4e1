// qg_layer.cu -- the operators around attention in a decoder layer: norms before and after a
// block fused with its gate and residual scale (qg_norm_residual), and rotary positions with
// the append to the paged cache (qg_rope_append, qg_rope_turns).
#include <algorithm>
#include <cmath>

#include "../../include/qg.h"
#include "qg_host.h"
#include "qg_types.cuh"

namespace qg {

// ----------------------------------------------------------------------------- residual norms
// Per row: t = y, optionally t <- t * rsqrt(mean(t^2) + eps) * (w_off + w_post), optionally
// t <- t * gate; r = res + alpha * t; x = r * rsqrt(mean(r^2) + eps) * (w_off + w_pre).
// Everything is fp32 between the loads and the one rounding of each output; x is formed from
// the unrounded r.  Bound by memory: each input is read once and each output written once,
// the row staying in registers between the two reductions.  4096 rows of 5120 (fp32 with gate
// and residual, bf16 out): 59.4 us, 0.94 of the measured copy bandwidth; one row: 5 us a call, 3.0 in a
// graph, the launch and two reductions.  Rows off the vector boundary take loads of one element: 4096 rows of
// 5121, fp32, 145 us (0.34), against 50 for 5120.
struct NormArgs {
    const void *y, *res, *gate;
    const float *w_post, *w_pre;
    void *res_out, *x_out;
    int64_t ldy, ldres, ldgate;  // elements between rows (ldgate 0: one row for all)
    float w_off, alpha, eps;
    int M, H;
    int tpr;  // threads per row (a multiple of 32)
};

// Sum over the threads of a row; `red` holds one value per warp of the block.  Two buffers
// alternate, so one barrier per sum is enough.
__device__ __forceinline__ float row_sum(float v, float *red, int warp, int w0, int nw) {
    v = warp_sum(v);
    if (nw == 1) return v;
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return warp_sum(lane < nw ? red[w0 + lane] : 0.0f);
}

// A thread holds NV groups of VEC consecutive elements, tpr groups apart.
template <class Y, class R, class X, int VEC, int NV>
__global__ void __launch_bounds__(1024) norm_residual_kernel(const NormArgs a) {
    __shared__ float red[2][32];
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5;
    const int nw = a.tpr >> 5, rg = warp / nw, w0 = rg * nw;
    const unsigned row = blockIdx.x * (blockDim.x / a.tpr) + rg;  // the last block's may pass 2^31
    const bool live = row < (unsigned)a.M;
    const int i0 = (threadIdx.x - w0 * 32) * VEC, step = a.tpr * VEC;
    const Y *y = static_cast<const Y *>(a.y) + (int64_t)(live ? row : 0) * a.ldy;
    const Y *gate = a.gate ? static_cast<const Y *>(a.gate) + (int64_t)(live ? row : 0) * a.ldgate : nullptr;
    const R *res = a.res ? static_cast<const R *>(a.res) + (int64_t)(live ? row : 0) * a.ldres : nullptr;
    const float inv = 1.0f / (float)a.H;

    // places past the row's end load its start and count as zero: a load under a branch would be
    // waited for there
    float t[NV][VEC], r[NV][VEC] = {};
#pragma unroll
    for (int j = 0; j < NV; ++j) load_vec<Y, VEC>(y + (i0 + j * step < a.H ? i0 + j * step : 0), t[j]);
    if (res) {
#pragma unroll
        for (int j = 0; j < NV; ++j) load_vec<R, VEC>(res + (i0 + j * step < a.H ? i0 + j * step : 0), r[j]);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (i0 + j * step >= a.H) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) t[j][e] = r[j][e] = 0.0f;
        }
    if (a.w_post) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) s = fmaf(t[j][e], t[j][e], s);
        const float k = rsqrtf(row_sum(s, red[0], warp, w0, nw) * inv + a.eps);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float w[VEC];
            load_vec<float, VEC>(a.w_post + (i0 + j * step < a.H ? i0 + j * step : 0), w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) t[j][e] = t[j][e] * k * (a.w_off + w[e]);
        }
    }
    if (gate) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float g[VEC];
            load_vec<Y, VEC>(gate + (i0 + j * step < a.H ? i0 + j * step : 0), g);
#pragma unroll
            for (int e = 0; e < VEC; ++e) t[j][e] = i0 + j * step < a.H ? t[j][e] * g[e] : 0.0f;
        }
    }
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = i0 + j * step;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            r[j][e] = fmaf(a.alpha, t[j][e], r[j][e]);
            s = fmaf(r[j][e], r[j][e], s);
        }
        if (live && i < a.H && a.res_out) store_vec<R, VEC>(static_cast<R *>(a.res_out) + (int64_t)row * a.H + i, r[j]);
    }
    if (!a.x_out) return;
    const float k = rsqrtf(row_sum(s, red[1], warp, w0, nw) * inv + a.eps);
    if (!live) return;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = i0 + j * step;
        if (i < a.H) {
            float w[VEC];
            load_vec<float, VEC>(a.w_pre + i, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) r[j][e] = r[j][e] * k * (a.w_off + w[e]);
            store_vec<X, VEC>(static_cast<X *>(a.x_out) + (int64_t)row * a.H + i, r[j]);
        }
    }
}

constexpr int NORM_MAX_H = 16384;  // 1024 threads x 16 elements of y and of r in registers

template <class Y, class R, class X, int VEC, int NV>
static int norm_launch(NormArgs a, cudaStream_t s) {
    const int per = VEC * NV;
    a.tpr = (((a.H + per - 1) / per) + 31) / 32 * 32;
    const int rpb = a.tpr >= 256 ? 1 : 256 / a.tpr;  // short rows share a block
    return launch_programmatic(norm_residual_kernel<Y, R, X, VEC, NV>, dim3(((unsigned)a.M + rpb - 1) / rpb), rpb * a.tpr,
                               0, s, a)
               ? QG_OK
               : QG_ECUDA;
}
template <class Y, class R, class X>
static int norm_run(const NormArgs &a, bool vec, cudaStream_t s) {
    if (!vec) return a.H <= 4096 ? norm_launch<Y, R, X, 1, 4>(a, s) : norm_launch<Y, R, X, 1, 16>(a, s);
    return a.H <= 512 ? norm_launch<Y, R, X, 4, 1>(a, s) : norm_launch<Y, R, X, 4, 4>(a, s);
}
template <class Y, class R>
static int norm_x(const NormArgs &a, int x_type, bool vec, cudaStream_t s) {
    switch (x_type) {
    case QG_F32: return norm_run<Y, R, float>(a, vec, s);
    case QG_F16: return norm_run<Y, R, f16>(a, vec, s);
    default: return norm_run<Y, R, bf16>(a, vec, s);
    }
}

// ----------------------------------------------------------------------------- rotary positions
// The phase of pair j at position p is p * turns[j] mod 2^64 in units of 2^-64 turns: whole
// turns drop out of the 64-bit product exactly, so the angle is as exact at position 2^30
// as at 1 and no table of positions is read.  The upper 32 bits, as a fraction of a turn in
// [-1/2, 1/2), go to sincospi.
//
// One warp takes one token and a run of its heads: the sines of the token are computed once
// and used for all of them.  A lane holds both elements of its pairs, four pairs of one head, so
// that rotating exchanges nothing between lanes and 32 / (D / 8) heads share an instruction
// (rope_quads_kernel); 4096 tokens of 32 + 2 x 8 heads of 128, fp32 to an 8-bit cache: 30 us
// (0.70 of the measured copy bandwidth; to fp16 26.3 us, 0.85), with 8 to 16 heads a warp 33, with
// more warps resident and fewer registers 37.  To 8 bits each lane quantizes its elements in every grouping
// (blocks in 4 lanes, two runs in 8) and keeps the one that holds, so that no lane branches.
// Rotated parts that are no multiple of 8 elements (64 for the keys of an 8-bit cache in halves,
// whose blocks of 32 must not straddle), and heads of 64 off a boundary of 4 elements, take
// rope_append_kernel: D / 32 consecutive elements per
// lane, partners from other lanes; the same with 96 (100) elements rotated in halves 39 (45) us.  The first is
// bound by memory for many tokens; one token is a launch and two loads deep (4.7 us a call, 3.1 in a
// graph).
struct RopeArgs {
    const void *q, *k, *v;
    int64_t ldq, hdq, ldk, hdk, ldv, hdv;  // elements between tokens, between heads
    const unsigned long long *turns;
    const float *wq, *wk;
    void *q_out;
    void *kc, *vc, *kd, *vd;
    int64_t page_stride, head_stride, slot_stride, step_stride;  // elements of the pools
    Batch bt;
    int Hq, Hk, rot, pairs;
    int hpw;  // heads per warp
    bool runs4;  // every head of q, k and v starts on a boundary of 4 elements
    float amp, eps;
};

// The sequence that new token t belongs to (the last b with q_start[b] <= t): 32 probes a step.
__device__ __forceinline__ int token_seq(const Batch &bt, int t, int lane) {
    int lo = 0, n = bt.batch;  // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int at = lo + lane * step;
        const unsigned m = __ballot_sync(0xffffffffu, lane * step < n && (lane == 0 || bt.q_start[at] <= t));
        // q_start does not decrease, so the set lanes are the first ones; otherwise any answer is in range
        const int last = __popc(m) - 1;
        lo += last * step;
        n = min(step, n - last * step);
    }
    return lo;
}

// The larger one; NaN where one is (fmaxf would drop it, and the cache would read finite).
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

constexpr int ROPE_WARPS = 4;
constexpr int ROPE_U = 2;  // heads whose loads are in flight together

template <class I, int C, int EPL>
__global__ void __launch_bounds__(ROPE_WARPS * 32, EPL == 8 ? 5 : 8) rope_append_kernel(const RopeArgs a) {
    using Q = typename CacheT<C>::Q;
    constexpr int D = EPL * 32;
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int heads = a.Hq + 2 * a.Hk, groups = (heads + a.hpw - 1) / a.hpw;
    const int64_t item = (int64_t)blockIdx.x * ROPE_WARPS + (threadIdx.x >> 5);
    if (item >= (int64_t)a.bt.tokens * groups) return;
    const int t = (int)(item / groups), h0 = (int)(item % groups) * a.hpw, h1 = min(heads, h0 + a.hpw);

    const int b = token_seq(a.bt, t, lane);
    const Seq sq = seq_of(a.bt, b);
    const int pos = sq.len - sq.n + (t - sq.first);
    const bool valid = t >= sq.first && t < sq.first + sq.n && pos >= 0;
    int page = -1, slot = 0;
    if (valid) {
        page = a.bt.pages[b * a.bt.table_stride + pos / a.bt.page];
        slot = pos % a.bt.page;
        if (page >= a.bt.n_pages) page = -1;
    }

    const int e0 = lane * EPL, half = a.rot / 2;
    const bool near = !a.pairs && half % EPL == 0;  // a pair's two elements sit at one place of two lanes
    float cs[EPL], sn[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        cs[i] = 1.0f;
        sn[i] = 0.0f;
        const int e = e0 + i;
        if (e < a.rot && h0 < a.Hq + a.Hk) {
            const int j = a.pairs ? e >> 1 : (e < half ? e : e - half);
            const unsigned long long ph = (unsigned long long)(long long)pos * a.turns[j];
            float s, c;
            sincospif((float)(int)(ph >> 32) * 0x1p-31f, &s, &c);
            cs[i] = c * a.amp;
            // x_e' = x_e cos -+ partner sin: minus for the first of a pair
            sn[i] = (a.pairs ? (e & 1) == 0 : e < half) ? -s * a.amp : s * a.amp;
        }
    }

    for (int hb = h0; hb < h1; hb += ROPE_U) {
        float x[ROPE_U][EPL];
        const I *src[ROPE_U];
#pragma unroll
        for (int u = 0; u < ROPE_U; ++u) {
            const int h = min(hb + u, h1 - 1);
            src[u] = h < a.Hq            ? static_cast<const I *>(a.q) + (int64_t)t * a.ldq + (int64_t)h * a.hdq
                     : h < a.Hq + a.Hk ? static_cast<const I *>(a.k) + (int64_t)t * a.ldk + (int64_t)(h - a.Hq) * a.hdk
                                         : static_cast<const I *>(a.v) + (int64_t)t * a.ldv +
                                               (int64_t)(h - a.Hq - a.Hk) * a.hdv;
            load_vec<I, EPL>(src[u] + e0, x[u]);
        }
#pragma unroll
        for (int u = 0; u < ROPE_U; ++u) {
            const int h = hb + u;
            if (h >= h1) break;
            const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hk;
            const float *w = is_q ? a.wq : a.wk;
            float k = 1.0f;
            if (!is_v) {
                if (w) {
                    float s = 0.0f;
#pragma unroll
                    for (int i = 0; i < EPL; ++i) s = fmaf(x[u][i], x[u][i], s);
                    k = rsqrtf(warp_sum(s) * (1.0f / D) + a.eps);
#pragma unroll
                    for (int i = 0; i < EPL; ++i) x[u][i] = x[u][i] * k * w[e0 + i];
                }
                float p[EPL];
                if (a.pairs) {
#pragma unroll
                    for (int i = 0; i < EPL; ++i) p[i] = x[u][i ^ 1];
                } else if (near) {
                    const int d = half / EPL, other = e0 < half ? lane + d : e0 < a.rot ? lane - d : lane;
#pragma unroll
                    for (int i = 0; i < EPL; ++i) p[i] = __shfl_sync(0xffffffffu, x[u][i], other);
                } else {  // the pair straddles places: fetch the partner again
#pragma unroll
                    for (int i = 0; i < EPL; ++i) {
                        const int e = e0 + i, o = e < half ? e + half : e < a.rot ? e - half : e;
                        p[i] = to_f32(src[u][o]) * k * (w ? w[o] : 1.0f);
                    }
                }
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (e0 + i < a.rot) x[u][i] = fmaf(p[i], sn[i], x[u][i] * cs[i]);
            }
            if (is_q) {
                if (!valid) {
#pragma unroll
                    for (int i = 0; i < EPL; ++i) x[u][i] = 0.0f;
                }
                store_vec<Q, EPL>(static_cast<Q *>(a.q_out) + ((int64_t)t * a.Hq + h) * D + e0, x[u]);
                continue;
            }
            if (page < 0) continue;
            const int kh = is_v ? h - a.Hq - a.Hk : h - a.Hq;
            const int64_t at = page * a.page_stride + kh * a.head_stride + slot * a.slot_stride + e0;
            void *pool = is_v ? a.vc : a.kc;
            if constexpr (C != CACHE_Q8) {
                store_vec<Q, EPL>(static_cast<Q *>(pool) + at, x[u]);
            } else {
                // the Q8_0 rule: step = amax / 127 per 32 elements, codes by the unrounded step
                float m = 0.0f;
#pragma unroll
                for (int i = 0; i < EPL; ++i) m = max_nan(m, fabsf(x[u][i]));
#pragma unroll
                for (int o = 16 / EPL; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                const float d = __fdiv_rn(m, 127.0f), id = m > 0.0f ? __fdividef(127.0f, m) : 0.0f;
                uint32_t c[(EPL + 3) / 4] = {};
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const int code = max(-127, min(127, __float2int_rn(x[u][i] * id)));
                    c[i / 4] |= ((uint32_t)code & 0xffu) << (8 * (i % 4));
                }
                int8_t *dst = static_cast<int8_t *>(pool) + at;
                if constexpr (EPL == 2)
                    *reinterpret_cast<uint16_t *>(dst) = (uint16_t)c[0];
                else if constexpr (EPL == 4)
                    *reinterpret_cast<uint32_t *>(dst) = c[0];
                else
                    *reinterpret_cast<uint2 *>(dst) = make_uint2(c[0], c[1]);
                if (lane % (32 / EPL) == 0)
                    (static_cast<f16 *>(is_v ? a.vd : a.kd) + page * a.step_stride +
                     ((int64_t)kh * a.bt.page + slot) * (D / 32))[e0 / 32] =
                        __float2half_rn(d);
            }
        }
    }
}

// Codes and step of a block whose elements are spread over LANES neighbouring lanes: the Q8_0 rule.
template <int LANES, int N>
__device__ __forceinline__ void quant_q8(const float (&x)[N], uint32_t (&c)[N / 4], float &d) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) m = max_nan(m, fabsf(x[i]));
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    d = __fdiv_rn(m, 127.0f);
    const float id = m > 0.0f ? __fdividef(127.0f, m) : 0.0f;
#pragma unroll
    for (int w = 0; w < N / 4; ++w) {
        c[w] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c[w] |= ((uint32_t)max(-127, min(127, __float2int_rn(x[4 * w + i] * id))) & 0xffu) << (8 * i);
    }
}

// A lane's 8 elements of a head are two runs of 4 at e[0] and e[1]: four pairs (the runs half apart, or
// adjacent with interleaved pairs), or 8 elements that pass through.
template <class I, int C, int D>
__global__ void __launch_bounds__(ROPE_WARPS * 32) rope_quads_kernel(const RopeArgs a) {
    using Q = typename CacheT<C>::Q;
    constexpr int LPH = D / 8, HPI = 32 / LPH;  // lanes of a head, heads of a step
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, c = lane % LPH, sub = lane / LPH;
    const int heads = a.Hq + 2 * a.Hk, groups = (heads + a.hpw - 1) / a.hpw;
    const int64_t item = (int64_t)blockIdx.x * ROPE_WARPS + (threadIdx.x >> 5);
    if (item >= (int64_t)a.bt.tokens * groups) return;
    const int t = (int)(item / groups), h0 = (int)(item % groups) * a.hpw, h1 = min(heads, h0 + a.hpw);

    const int b = token_seq(a.bt, t, lane);
    const Seq sq = seq_of(a.bt, b);
    const int pos = sq.len - sq.n + (t - sq.first);
    const bool valid = t >= sq.first && t < sq.first + sq.n && pos >= 0;
    int page = -1, slot = 0;
    if (valid) {
        page = a.bt.pages[b * a.bt.table_stride + pos / a.bt.page];
        slot = pos % a.bt.page;
        if (page >= a.bt.n_pages) page = -1;
    }

    const int half = a.rot / 2;
    const bool turns = 8 * c < a.rot;                       // the lane's elements are pairs
    const bool split = !a.pairs && turns;                   // runs `half` apart
    const int e0 = split ? 4 * c : 8 * c, e1 = split ? half + 4 * c : 8 * c + 4;
    float cs[4] = {1.0f, 1.0f, 1.0f, 1.0f}, sn[4] = {};
    if (turns && h0 < a.Hq + a.Hk) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned long long ph = (unsigned long long)(long long)pos * a.turns[4 * c + i];
            sincospif((float)(int)(ph >> 32) * 0x1p-31f, &sn[i], &cs[i]);
            cs[i] *= a.amp;
            sn[i] *= a.amp;
        }
    }
    const I *bq = static_cast<const I *>(a.q) + (int64_t)t * a.ldq, *bk = static_cast<const I *>(a.k) + (int64_t)t * a.ldk;
    const I *bv = static_cast<const I *>(a.v) + (int64_t)t * a.ldv;
    Q *qo = static_cast<Q *>(a.q_out) + (int64_t)t * a.Hq * D;
    const int64_t place = page * a.page_stride + slot * a.slot_stride, steps = page * a.step_stride + (int64_t)slot * (D / 32);

    for (int hb = h0; hb < h1; hb += HPI * ROPE_U) {
        float x[ROPE_U][8];
#pragma unroll
        for (int u = 0; u < ROPE_U; ++u) {
            const int h = min(hb + u * HPI + sub, h1 - 1);
            const bool is_v = h >= a.Hq + a.Hk;
            const I *src = h < a.Hq ? bq + h * a.hdq : is_v ? bv + (h - a.Hq - a.Hk) * a.hdv : bk + (h - a.Hq) * a.hdk;
            float lo[4], hi[4];
            load_vec<I, 4>(src + (is_v ? 8 * c : e0), lo);
            load_vec<I, 4>(src + (is_v ? 8 * c + 4 : e1), hi);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[u][i] = lo[i], x[u][4 + i] = hi[i];
        }
#pragma unroll
        for (int u = 0; u < ROPE_U; ++u) {
            if (hb + u * HPI >= h1) break;  // whole warp
            const int hh = hb + u * HPI + sub, h = min(hh, h1 - 1);
            const bool live = hh < h1, is_q = h < a.Hq, is_v = h >= a.Hq + a.Hk;
            const float *w = is_q ? a.wq : a.wk;
            if (a.wq || a.wk) {
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) s = fmaf(x[u][i], x[u][i], s);
#pragma unroll
                for (int o = LPH / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                if (w && !is_v) {
                    const float k = rsqrtf(s * (1.0f / D) + a.eps);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[u][i] *= k * w[e0 + i];
                        x[u][4 + i] *= k * w[e1 + i];
                    }
                }
            }
            if (turns && !is_v) {
                if (a.pairs) {  // pairs 0..3: elements (0, 1), (2, 3), ...
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p = x[u][2 * i], q = x[u][2 * i + 1];
                        x[u][2 * i] = fmaf(-q, sn[i], p * cs[i]);
                        x[u][2 * i + 1] = fmaf(p, sn[i], q * cs[i]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p = x[u][i], q = x[u][4 + i];
                        x[u][i] = fmaf(-q, sn[i], p * cs[i]);
                        x[u][4 + i] = fmaf(p, sn[i], q * cs[i]);
                    }
                }
            }
            const float lo[4] = {x[u][0], x[u][1], x[u][2], x[u][3]}, hi[4] = {x[u][4], x[u][5], x[u][6], x[u][7]};
            if (is_q) {
                if (live) {
                    const float zero[4] = {};
                    store_vec<Q, 4>(qo + h * D + e0, valid ? lo : zero);
                    store_vec<Q, 4>(qo + h * D + e1, valid ? hi : zero);
                }
            }
            // Lanes of queries that share a step with keys stay: the shuffles below are the whole warp's
            if (min(hb + u * HPI + HPI, h1) <= a.Hq) continue;  // whole warp
            const int kh = is_v ? h - a.Hq - a.Hk : h - a.Hq, f0 = is_v ? 8 * c : e0, f1 = is_v ? 8 * c + 4 : e1;
            const bool keep = live && !is_q && page >= 0;
            if constexpr (C != CACHE_Q8) {
                if (keep) {
                    Q *dst = static_cast<Q *>(is_v ? a.vc : a.kc) + place + kh * a.head_stride;
                    store_vec<Q, 4>(dst + f0, lo);
                    store_vec<Q, 4>(dst + f1, hi);
                }
            } else {
                // values, interleaved pairs and elements that pass through: blocks of 32 in 4 lanes; halves: the
                // first runs of 8 lanes are one block, their second runs another
                uint32_t cd[2], c0[1], c1[1];
                float d, d0, d1;
                quant_q8<4>(x[u], cd, d);
                quant_q8<8>(lo, c0, d0);
                quant_q8<8>(hi, c1, d1);
                const bool halves = split && !is_v;
                if (keep) {
                    int8_t *dst = static_cast<int8_t *>(is_v ? a.vc : a.kc) + place + kh * a.head_stride;
                    f16 *st = static_cast<f16 *>(is_v ? a.vd : a.kd) + steps + (int64_t)kh * a.bt.page * (D / 32);
                    *reinterpret_cast<uint32_t *>(dst + f0) = halves ? c0[0] : cd[0];
                    *reinterpret_cast<uint32_t *>(dst + f1) = halves ? c1[0] : cd[1];
                    if (halves) {
                        if (c % 8 == 0) st[f0 / 32] = __float2half_rn(d0), st[f1 / 32] = __float2half_rn(d1);
                    } else if (c % 4 == 0) {
                        st[f0 / 32] = __float2half_rn(d);
                    }
                }
            }
        }
    }
}

template <class I, int C, int EPL>
static int rope_launch(const RopeArgs &a, int64_t warps, cudaStream_t s) {
    const bool quads = a.runs4 && a.rot % 8 == 0 && (C != CACHE_Q8 || a.pairs || a.rot % 64 == 0);
    return launch_programmatic(quads ? rope_quads_kernel<I, C, EPL * 32> : rope_append_kernel<I, C, EPL>,
                               dim3((unsigned)((warps + ROPE_WARPS - 1) / ROPE_WARPS)), ROPE_WARPS * 32, 0, s, a)
               ? QG_OK
               : QG_ECUDA;
}
template <class I, int C>
static int rope_dim(const RopeArgs &a, int D, int64_t warps, cudaStream_t s) {
    return D == 64 ? rope_launch<I, C, 2>(a, warps, s) : D == 128 ? rope_launch<I, C, 4>(a, warps, s) : rope_launch<I, C, 8>(a, warps, s);
}
template <class I>
static int rope_cache(const RopeArgs &a, int type, int D, int64_t warps, cudaStream_t s) {
    return type == QG_F16    ? rope_dim<I, CACHE_F16>(a, D, warps, s)
           : type == QG_BF16 ? rope_dim<I, CACHE_BF16>(a, D, warps, s)
                             : rope_dim<I, CACHE_Q8>(a, D, warps, s);
}

static bool float_type(int t) { return t == QG_F32 || t == QG_F16 || t == QG_BF16; }
static int type_size(int t) { return t == QG_F32 ? 4 : 2; }

}  // namespace qg

using namespace qg;

extern "C" {

int qg_norm_residual(const void *y, int y_type, int64_t ldy, const void *res, int res_type, int64_t ldres,
                     const float *w_post, const void *gate, int64_t ldgate, const float *w_pre, float w_offset,
                     float alpha, float eps, void *res_out, void *x_out, int x_type, int M, int H, void *stream) {
    if (!y || (!res_out && !x_out) || M < 1 || H < 1 || H > NORM_MAX_H || !float_type(y_type) || !float_type(x_type))
        return QG_EINVAL;
    if (res_type != QG_F32 && res_type != y_type) return QG_EINVAL;
    if (ldy < H || (res && ldres < H) || (gate && ldgate != 0 && ldgate < H) || (x_out && !w_pre) || !(eps >= 0.0f))
        return QG_EINVAL;
    if (res && res_out == res && ldres != H && M > 1) return QG_EINVAL;
    const int ys = type_size(y_type), rs = type_size(res_type), xs = type_size(x_type);
    if (!host_aligned(y, ys) || !host_aligned(res, rs) || !host_aligned(gate, ys) || !host_aligned(res_out, rs) ||
        !host_aligned(x_out, xs) || !host_aligned(w_post, 4) || !host_aligned(w_pre, 4))
        return QG_EALIGN;
    const int sms = device_sms();
    if (sms < 0) return sms;
    // four elements a load where every row starts on such a boundary
    const bool vec = H % 4 == 0 && ldy % 4 == 0 && (!res || ldres % 4 == 0) && (!gate || ldgate % 4 == 0) &&
                     host_aligned(y, 4 * ys) && host_aligned(res, 4 * rs) && host_aligned(gate, 4 * ys) &&
                     host_aligned(res_out, 4 * rs) && host_aligned(x_out, 4 * xs) && host_aligned(w_post, 16) &&
                     host_aligned(w_pre, 16);
    NormArgs a{y, res, gate, w_post, w_pre, res_out, x_out, ldy, ldres, ldgate, w_offset, alpha, eps, M, H, 0};
    cudaStream_t s = (cudaStream_t)stream;
    switch (y_type) {
    case QG_F32: return norm_x<float, float>(a, x_type, vec, s);
    case QG_F16: return res_type == QG_F32 ? norm_x<f16, float>(a, x_type, vec, s) : norm_x<f16, f16>(a, x_type, vec, s);
    default: return res_type == QG_F32 ? norm_x<bf16, float>(a, x_type, vec, s) : norm_x<bf16, bf16>(a, x_type, vec, s);
    }
}

int qg_rope_turns(int rot, double base, int scaling, double factor, double original, double beta_fast, double beta_slow,
                  uint64_t *turns, float *amp) {
    if (!turns || rot < 2 || rot % 2 || !(base > 1.0) || scaling < QG_ROPE_PLAIN || scaling > QG_ROPE_YARN) return QG_EINVAL;
    if (scaling != QG_ROPE_PLAIN && !(factor >= 1.0)) return QG_EINVAL;
    if (scaling == QG_ROPE_YARN && (!(original >= 1.0) || !(beta_fast > 0.0) || !(beta_slow > 0.0))) return QG_EINVAL;
    if (scaling == QG_ROPE_NTK && rot < 4) return QG_EINVAL;
    const int half = rot / 2;
    const double two_pi = 6.283185307179586476925286766559;
    if (scaling == QG_ROPE_NTK) base *= std::pow(factor, (double)rot / (rot - 2));
    double lo = 0, hi = 0;
    if (scaling == QG_ROPE_YARN) {
        const double per = half / std::log(base);
        lo = std::fmax(std::floor(per * std::log(original / (beta_fast * two_pi))), 0.0);
        hi = std::fmin(std::ceil(per * std::log(original / (beta_slow * two_pi))), rot - 1.0);  // the ramp may end past the last pair
    }
    for (int j = 0; j < half; ++j) {
        const double f = std::pow(base, -(double)j / half);
        double g = f;
        if (scaling == QG_ROPE_LINEAR) g = f / factor;
        if (scaling == QG_ROPE_YARN) {
            const double ramp = std::fmin(std::fmax((j - lo) / std::fmax(hi - lo, 1e-3), 0.0), 1.0);
            g = f / factor * ramp + f * (1.0 - ramp);
        }
        // f <= 1 radian per position, so the fraction of a turn is below 2^64 as it stands
        turns[j] = (uint64_t)std::floor(std::ldexp(g / two_pi, 64));
    }
    if (amp) *amp = scaling == QG_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
    return QG_OK;
}

int qg_rope_append(const void *q, int64_t ldq, int64_t hdq, const void *k, int64_t ldk, int64_t hdk, const void *v,
                   int64_t ldv, int64_t hdv, int in_type, int tokens, int q_heads, const uint64_t *turns, int rot, int pairs,
                   float amp, const float *wq, const float *wk, float eps, void *q_out, const qg_paged *cache,
                   void *stream) {
    if (!q || !k || !v || !q_out || !cache || !float_type(in_type) || tokens < 1 || q_heads < 1) return QG_EINVAL;
    if (const int rc = paged_check(*cache)) return rc;
    const int D = cache->dim, Hk = cache->kv_heads;
    if (rot < 0 || rot > D || rot % 2 || (rot && !turns) || !(eps >= 0.0f) || q_heads % Hk) return QG_EINVAL;
    if ((int64_t)tokens * (q_heads + 2 * (int64_t)Hk) > INT32_MAX) return QG_EINVAL;
    if (hdq < D || hdk < D || hdv < D || ldq < D || ldk < D || ldv < D) return QG_EINVAL;
    const int es = type_size(in_type);
    const size_t va = (size_t)std::min(16, D / 32 * es);  // bytes of one lane's load
    for (const void *p : {q, k, v})
        if (!host_aligned(p, va)) return QG_EALIGN;
    for (const int64_t n : {ldq, hdq, ldk, hdk, ldv, hdv})
        if ((size_t)(n * es) % va) return QG_EALIGN;
    if (!host_aligned(q_out, 16) || !host_aligned(turns, 8) || !host_aligned(wq, 4) || !host_aligned(wk, 4)) return QG_EALIGN;
    const int sms = device_sms();
    if (sms < 0) return sms;
    RopeArgs a{};
    a.q = q, a.k = k, a.v = v;
    a.ldq = ldq, a.hdq = hdq, a.ldk = ldk, a.hdk = hdk, a.ldv = ldv, a.hdv = hdv;
    a.turns = reinterpret_cast<const unsigned long long *>(turns);
    a.wq = wq, a.wk = wk;
    a.q_out = q_out;
    a.kc = cache->k, a.vc = cache->v, a.kd = cache->kd, a.vd = cache->vd;
    a.page_stride = cache->page_stride, a.head_stride = cache->head_stride, a.slot_stride = cache->slot_stride;
    a.step_stride = cache->step_stride;
    a.bt = paged_batch(*cache, tokens);
    a.Hq = q_heads, a.Hk = Hk, a.rot = rot, a.pairs = pairs != 0;
    a.runs4 = true;
    for (const void *p : {q, k, v}) a.runs4 = a.runs4 && host_aligned(p, 4 * es);
    for (const int64_t n : {ldq, hdq, ldk, hdk, ldv, hdv}) a.runs4 = a.runs4 && n % 4 == 0;
    a.amp = amp, a.eps = eps;
    // few tokens: a warp takes as many heads as it has room for in one step (latency); many: up to 24
    // share the sines, as long as the warps fill the machine
    const int heads = q_heads + 2 * Hk, step = 256 / D;
    const int64_t items = (int64_t)tokens * heads, fill = (int64_t)sms * 32;
    a.hpw = (int)std::min<int64_t>(std::max<int64_t>(items / fill / step, 1) * step, 24);
    const int64_t warps = (int64_t)tokens * ((heads + a.hpw - 1) / a.hpw);
    cudaStream_t s = (cudaStream_t)stream;
    switch (in_type) {
    case QG_F32: return rope_cache<float>(a, cache->type, D, warps, s);
    case QG_F16: return rope_cache<f16>(a, cache->type, D, warps, s);
    default: return rope_cache<bf16>(a, cache->type, D, warps, s);
    }
}

}  // extern "C"
