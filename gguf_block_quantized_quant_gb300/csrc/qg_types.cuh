// qg_types.cuh -- element types of the decoder-layer operators (fp32, fp16, bf16) and the
// paged cache they share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/qg.h"
#include "qg_common.cuh"
#include "qg_host.h"

namespace qg {

using f16 = __half;
using bf16 = __nv_bfloat16;

template <class T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<f16>(f16 x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f32<bf16>(bf16 x) { return __bfloat162float(x); }

// Nearest value of T, ties to even.
template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ f16 from_f32<f16>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ bf16 from_f32<bf16>(float x) { return __float2bfloat16_rn(x); }

// Two values packed in one register, a in the low half.
template <class T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<f16>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<bf16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <class T>
__device__ __forceinline__ float2 unpack2(uint32_t v);
template <>
__device__ __forceinline__ float2 unpack2<f16>(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}
template <>
__device__ __forceinline__ float2 unpack2<bf16>(uint32_t v) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v));
}

// Two fp32 values in a register pair, and the instructions on both.
__device__ __forceinline__ uint64_t pack_b32x2(uint32_t a, uint32_t b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint64_t pack_f32x2(float a, float b) { return pack_b32x2(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// N consecutive elements as fp32; N * sizeof(T) is a power of two and p is aligned to it
// (to 16 bytes where that is more).
template <class T, int N>
__device__ __forceinline__ void load_vec(const T *p, float (&v)[N]) {
    if constexpr (N == 1) {
        v[0] = to_f32(*p);
    } else {
        constexpr int BYTES = N * (int)sizeof(T);
        constexpr int W = BYTES / 4;
        uint32_t w[W];
        if constexpr (BYTES == 4) {
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        } else if constexpr (BYTES == 8) {
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            w[0] = u.x;
            w[1] = u.y;
        } else {
#pragma unroll
            for (int i = 0; i < W / 4; ++i) {
                const uint4 u = reinterpret_cast<const uint4 *>(p)[i];
                w[4 * i] = u.x;
                w[4 * i + 1] = u.y;
                w[4 * i + 2] = u.z;
                w[4 * i + 3] = u.w;
            }
        }
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float2 f = unpack2<T>(w[i]);
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
}
template <class T, int N>
__device__ __forceinline__ void store_vec(T *p, const float (&v)[N]) {
    if constexpr (N == 1) {
        *p = from_f32<T>(v[0]);
    } else {
        constexpr int BYTES = N * (int)sizeof(T);
        constexpr int W = BYTES / 4;
        uint32_t w[W];
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = __float_as_uint(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
        }
        if constexpr (BYTES == 4) {
            *reinterpret_cast<uint32_t *>(p) = w[0];
        } else if constexpr (BYTES == 8) {
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
            for (int i = 0; i < W / 4; ++i)
                reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
    }
}

// What the pools of a cache hold, and the type of the queries beside it.
enum { CACHE_F16, CACHE_BF16, CACHE_Q8 };
template <int C>
struct CacheT {
    using Q = f16;
};
template <>
struct CacheT<CACHE_BF16> {
    using Q = bf16;
};

// The sequences of one call, as the kernels read them (device arrays of the caller).
struct Batch {
    const int32_t *q_start;  // batch + 1: first new token of each sequence
    const int32_t *kv_len;   // batch: slots in use, the new tokens included
    const int32_t *pages;    // batch x table_stride: page ids in order
    int batch, table_width, page, n_pages, tokens;
    int64_t table_stride;
};

struct Seq {
    int first;  // first new token (row of q)
    int n;      // new tokens
    int len;    // slots in use
};

constexpr int64_t MAX_SLOTS = 0x7fffff00;  // of a sequence: a tile that holds its last slot ends below 2^31

// The sequence's lengths, held inside the caller's arrays: token rows inside [0, tokens), slots
// inside the page table (and below MAX_SLOTS).
__device__ __forceinline__ Seq seq_of(const Batch &bt, int b) {
    Seq s;
    s.first = min(max(bt.q_start[b], 0), bt.tokens);
    s.n = min(max(bt.q_start[b + 1], s.first), bt.tokens) - s.first;
    s.len = (int)min((int64_t)max(bt.kv_len[b], 0), min((int64_t)bt.table_width * bt.page, MAX_SLOTS));
    return s;
}

// Argument checks that every call with a cache makes (host).
inline int paged_check(const qg_paged &c) {
    if (c.type != QG_F16 && c.type != QG_BF16 && c.type != QG_Q8_0) return QG_EINVAL;
    const bool q8 = c.type == QG_Q8_0;
    if (c.kv_heads < 1 || (c.dim != 64 && c.dim != 128 && c.dim != 256) || c.page < 16 || c.page % 16 || c.n_pages < 1 ||
        c.batch < 1 || c.table_width < 1 || c.table_stride < c.table_width)
        return QG_EINVAL;
    if (!c.k || !c.v || !c.q_start || !c.kv_len || !c.pages || (q8 && (!c.kd || !c.vd))) return QG_EINVAL;
    if (c.slot_stride < c.dim || c.head_stride < c.dim || c.page_stride < c.dim) return QG_EINVAL;
    const int64_t steps = (int64_t)c.kv_heads * c.page * (c.dim / 32);
    if (q8 && c.step_stride < steps) return QG_EINVAL;
    const int per = q8 ? 16 : 8;  // elements of 16 bytes
    if (!host_aligned(c.k, 16) || !host_aligned(c.v, 16) || c.page_stride % per || c.head_stride % per || c.slot_stride % per)
        return QG_EALIGN;
    if (q8 && (!host_aligned(c.kd, 16) || !host_aligned(c.vd, 16) || c.step_stride % 8)) return QG_EALIGN;
    if (!host_aligned(c.q_start, 4) || !host_aligned(c.kv_len, 4) || !host_aligned(c.pages, 4)) return QG_EALIGN;
    return QG_OK;
}
inline Batch paged_batch(const qg_paged &c, int tokens) {
    return Batch{c.q_start, c.kv_len, c.pages, c.batch, c.table_width, c.page, c.n_pages, tokens, c.table_stride};
}

}  // namespace qg
