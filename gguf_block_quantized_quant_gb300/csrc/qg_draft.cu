// qg_draft.cu -- the operators around drafted tokens that are not attention: masks and positions of trees
// (qg_tree_masks), accepted drafts moved together in the cache (qg_cache_keep), and penalties, biases and
// grammar masks on the logits (qg_logits_adjust).
#include <algorithm>

#include "../../include/qg.h"
#include "qg_host.h"
#include "qg_types.cuh"

namespace qg {

// ----------------------------------------------------------------------------- masks of trees
// A block per sequence, the last block for rows of no sequence; a thread follows its draft's ancestors, whose indices
// fall, so that the words of its row are written once each, from the last down.  A launch and two dependent loads.
constexpr int TREE_MAX = 1024, TREE_THREADS = 256;

__global__ void __launch_bounds__(TREE_THREADS) tree_masks_kernel(const int32_t *parents, const int32_t *q_start, const int32_t *kv_len,
                                                                  int tokens, int batch, uint32_t *tree, int words, int32_t *positions) {
    __shared__ int16_t up[TREE_MAX];
    griddep_wait();
    griddep_launch_dependents();
    const int b = blockIdx.x;
    if (b == batch) {
        const int lo = min(max(q_start[0], 0), tokens), hi = min(max(q_start[batch], 0), tokens);
        for (int i = threadIdx.x; i < lo + tokens - hi; i += TREE_THREADS) {
            const int64_t t = i < lo ? i : hi + i - lo;
            positions[t] = 0;
            for (int w = 0; w < words; ++w) tree[t * words + w] = 0u;
        }
        return;
    }
    const int first = min(max(q_start[b], 0), tokens), n = min(max(q_start[b + 1], first), tokens) - first;
    const int base = max(kv_len[b], 0) - n, held = min(n, min(TREE_MAX, 32 * words));
    for (int i = threadIdx.x; i < held; i += TREE_THREADS) {
        const int p = parents[first + i];
        up[i] = (int16_t)(p >= 0 && p < i ? p : -1);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += TREE_THREADS) {
        uint32_t *row = tree + (int64_t)(first + i) * words;
        int depth = 0, w = words - 1;
        uint32_t bits = 0;
        for (int p = i < held ? i : -1; p >= 0; p = up[p]) {
            for (; w > p >> 5; --w) {
                row[w] = bits;
                bits = 0;
            }
            bits |= 1u << (p & 31);
            ++depth;
        }
        for (; w >= 0; --w) {
            row[w] = bits;
            bits = 0;
        }
        positions[first + i] = base + max(depth - 1, 0);
    }
}

// ----------------------------------------------------------------------------- accepted drafts
// A thread owns 16 bytes of every slot of a head (4 bytes of its steps) and moves them for all kept drafts in order,
// KEEP_U loads in flight.  Index i takes from keep[i] >= i only, so a place is never written before what is still to be
// read from it: within a thread in order, and no two threads meet at a byte.  A launch and four dependent loads (lengths,
// indices, pages, data); the bytes that move are few.
constexpr int KEEP_THREADS = 256, KEEP_MAX = 1024, KEEP_U = 8;

struct KeepArgs {
    Batch bt;
    const int32_t *keep, *keep_len;
    int64_t keep_stride;
    int width;
    int32_t *kv_out;  // NULL: written by a kernel of its own
    uint8_t *k, *v, *kd, *vd;
    int64_t layer, page_stride, head_stride, slot_stride;  // bytes
    int64_t step_layer, step_page;                         // bytes
    int heads, chunks, step_words;                         // 16-byte chunks of a head's slot, 4-byte words of its steps
};

__device__ __forceinline__ int kept_of(const KeepArgs &a, const Seq &s, int b) { return min(max(a.keep_len[b], 0), min(a.width, s.n)); }

__global__ void __launch_bounds__(KEEP_THREADS) cache_keep_kernel(const KeepArgs a) {
    __shared__ int4 move[KEEP_MAX];  // page and slot to read, page and slot to write (page -1: nothing)
    griddep_wait();
    griddep_launch_dependents();
    const int b = blockIdx.y, tid = threadIdx.x;
    const Seq s = seq_of(a.bt, b);
    const int m = kept_of(a, s, b), base = s.len - s.n;
    if (a.kv_out && blockIdx.x == 0 && blockIdx.z == 0 && tid == 0) a.kv_out[b] = max(base + m, 0);
    for (int i = tid; i < m; i += KEEP_THREADS) {
        const int from = a.keep[b * a.keep_stride + i];
        int4 x = make_int4(0, 0, -1, 0);
        if (from > i && from < s.n && base + i >= 0) {
            const int32_t *pages = a.bt.pages + b * a.bt.table_stride;
            x = make_int4(pages[(base + from) / a.bt.page], (base + from) % a.bt.page, pages[(base + i) / a.bt.page], (base + i) % a.bt.page);
            if ((unsigned)x.x >= (unsigned)a.bt.n_pages) x.x = -1;  // reads as zeros
            if ((unsigned)x.z >= (unsigned)a.bt.n_pages) x.z = -1;
        }
        move[i] = x;
    }
    __syncthreads();
    const int data = 2 * a.heads * a.chunks, items = data + 2 * a.heads * a.step_words;
    const int x = blockIdx.x * KEEP_THREADS + tid;
    if (x >= items) return;
    auto run = [&](auto zero, auto at) {  // at(page, slot): the thread's place there
        using V = decltype(zero);
        for (int i0 = 0; i0 < m; i0 += KEEP_U) {
            V v[KEEP_U];
#pragma unroll
            for (int u = 0; u < KEEP_U; ++u) {
                const int4 mv = move[min(i0 + u, m - 1)];
                v[u] = zero;
                if (mv.z >= 0 && mv.x >= 0) v[u] = *reinterpret_cast<const V *>(at(mv.x, mv.y));
            }
#pragma unroll
            for (int u = 0; u < KEEP_U; ++u) {
                const int4 mv = move[min(i0 + u, m - 1)];
                if (i0 + u < m && mv.z >= 0) *reinterpret_cast<V *>(at(mv.z, mv.w)) = v[u];
            }
        }
    };
    if (x < data) {
        const int c = x % a.chunks, h = x / a.chunks % a.heads;
        uint8_t *pool = (x < a.heads * a.chunks ? a.k : a.v) + blockIdx.z * a.layer + h * a.head_stride + 16 * c;
        run(make_uint4(0, 0, 0, 0), [&](int page, int slot) { return pool + page * a.page_stride + slot * a.slot_stride; });
    } else {
        const int y = x - data, w = y % a.step_words, h = y / a.step_words % a.heads;
        uint8_t *pool = (y < a.heads * a.step_words ? a.kd : a.vd) + blockIdx.z * a.step_layer + 4 * w;
        run(0u, [&](int page, int slot) { return pool + page * a.step_page + ((int64_t)h * a.bt.page + slot) * (4 * a.step_words); });
    }
}

// The lengths, where they go over those that the blocks above read.
__global__ void __launch_bounds__(KEEP_THREADS) keep_lengths_kernel(const KeepArgs a, int32_t *kv_out) {
    griddep_wait();
    griddep_launch_dependents();
    const int b = blockIdx.x * KEEP_THREADS + threadIdx.x;
    if (b >= a.bt.batch) return;
    const Seq s = seq_of(a.bt, b);
    kv_out[b] = max(s.len - s.n + kept_of(a, s, b), 0);
}

// ----------------------------------------------------------------------------- logits
// A block takes a segment of a few rows, one after the other.  It counts the ids of the segment that the row's history and drafts
// hold in shared memory (a word per id: the count, bit 31 for ids of the prompt) and notes the last bias entry of each
// id there; rows of one sequence share that, but for their drafts, which are added before a row and taken off after it.  The logits
// are on their way to registers meanwhile.  Whole numbers are added, so the order of the atomics changes nothing.
// Bound by memory: the logits are read and written once; what hides the chain of dependent loads before them (sequence,
// lengths, ids) are the other blocks of the SM.
struct LogitsArgs {
    const void *x;
    void *out;
    int64_t ld, ldo;  // elements
    int V, seg;       // seg: ids of a segment, a multiple of 128
    int rows, group;  // group: rows of a block
    int in_place, has_bias;
    qg_logits how;
};

constexpr int LOGITS_THREADS = 256, LOGITS_U = 4, LOGITS_SEG = LOGITS_THREADS * LOGITS_U * 4;

// Four elements as they come.
template <class T>
struct Raw4 {
    uint2 w;
    __device__ __forceinline__ void load(const T *p) { w = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ void set(int k, T x) { reinterpret_cast<T *>(&w)[k] = x; }
    __device__ __forceinline__ void get(float (&v)[4]) const {
        const float2 a = unpack2<T>(w.x), b = unpack2<T>(w.y);
        v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    }
};
template <>
struct Raw4<float> {
    float4 w;
    __device__ __forceinline__ void load(const float *p) { w = *reinterpret_cast<const float4 *>(p); }
    __device__ __forceinline__ void set(int k, float x) { reinterpret_cast<float *>(&w)[k] = x; }
    __device__ __forceinline__ void get(float (&v)[4]) const { v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w; }
};

template <class I, class O>
__global__ void __launch_bounds__(LOGITS_THREADS, 4) logits_kernel(const LogitsArgs a) {
    extern __shared__ __align__(16) uint32_t lg_smem[];
    uint32_t *count = lg_smem;
    uint32_t *mask = count + a.seg;       // seg / 32 words
    uint32_t *entry = mask + a.seg / 32;  // seg words, where there are biases
    const int tid = threadIdx.x;
    const int segs = (a.V + 3 + a.seg - 1) / a.seg;
    const int row0 = (int)(blockIdx.x / segs) * a.group, row1 = min(row0 + a.group, a.rows);
    const int p0 = (int)(blockIdx.x % segs) * a.seg;
    griddep_wait();
    griddep_launch_dependents();

    int held = -2, held_ids0 = 0;  // the sequence (-1: none) whose ids are counted, and the segment's first id then
    float rep = 1.0f, freq = 0.0f, pres = 0.0f;
    const float *bias = nullptr;
    for (int row = row0; row < row1; ++row) {
        const I *x = static_cast<const I *>(a.x) + row * a.ld;
        O *out = static_cast<O *>(a.out) + row * a.ldo;
        // Places of a row are counted from the boundary of 4 elements before its start in `out`; id v is at place v + lead
        const int lead = (int)((reinterpret_cast<uintptr_t>(out) / sizeof(O)) & 3);
        const bool vec = (reinterpret_cast<uintptr_t>(x) / sizeof(I) & 3) == lead;
        const int ids0 = p0 - lead;                 // the segment's first id (below 0 in the first)
        const int n = min(a.seg, a.V + lead - p0);  // places of it up to the row's end
        if (n <= 0) continue;                       // the last row's lead may need a segment that this one's does not
        const int s = a.how.seq ? a.how.seq[row] : row;
        const bool known = (unsigned)s < (unsigned)a.how.batch;
        const bool in_place = std::is_same<I, O>::value && a.in_place;
        auto whole = [&](int q) { return vec && ids0 + 4 * q >= 0 && 4 * q + 4 <= n; };
        auto fetch = [&](Raw4<I> &v, int q) {
            const int id = ids0 + 4 * q;
            if (whole(q)) {
                v.load(x + id);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) v.set(k, id + k >= 0 && 4 * q + k < n ? x[id + k] : from_f32<I>(0.0f));
            }
        };
        Raw4<I> v[LOGITS_U];
        if (!in_place) {
#pragma unroll
            for (int u = 0; u < LOGITS_U; ++u)
                if (4 * (tid + u * LOGITS_THREADS) < n) fetch(v[u], tid + u * LOGITS_THREADS);
        }
        if (a.how.allow) {
            const uint32_t *allow = a.how.allow + row * a.how.allow_stride;
            const int words = (a.V + 31) / 32;
            for (int i = tid; i < a.seg / 32; i += LOGITS_THREADS) {
                const int at = ids0 + 32 * i, w = at >> 5;  // at may be below 0
                const uint32_t lo = w >= 0 && w < words ? allow[w] : 0u, hi = w + 1 < words ? allow[w + 1] : 0u;
                mask[i] = __funnelshift_r(lo, hi, at & 31);
            }
        }
        auto place = [&](int id) { return (unsigned)id < (unsigned)a.V ? id - ids0 : -1; };
        const bool fresh = (known ? s : -1) != held || ids0 != held_ids0;
        if (fresh) {
            held = known ? s : -1;
            held_ids0 = ids0;
            for (int i = tid; i < a.seg / 4; i += LOGITS_THREADS) reinterpret_cast<uint4 *>(count)[i] = make_uint4(0, 0, 0, 0);
            if (a.has_bias)
                for (int i = tid; i < a.seg / 4; i += LOGITS_THREADS) reinterpret_cast<uint4 *>(entry)[i] = make_uint4(0, 0, 0, 0);
            rep = 1.0f, freq = pres = 0.0f;
            int len = 0, said = 0, start = 0, entries = 0;
            if (known) {
                if (a.how.repetition) rep = a.how.repetition[s];
                if (a.how.frequency) freq = a.how.frequency[s];
                if (a.how.presence) pres = a.how.presence[s];
                if (a.how.history) {
                    len = min(max(a.how.history_len[s], 0), min(a.how.history_width, 1 << 30));
                    said = a.how.prompt_len ? a.how.prompt_len[s] : 0;
                }
                if (a.has_bias) {
                    start = min(max(a.how.bias_start[s], 0), a.how.bias_entries);
                    entries = min(a.how.bias_start[s + 1], a.how.bias_entries) - start;
                    bias = a.how.bias + start;
                }
            }
            __syncthreads();
            const int32_t *h = a.how.history + s * a.how.history_stride;
            auto add = [&](int id, int i) {
                const int at = place(id);
                if ((unsigned)at >= (unsigned)n) return;
                if (i < said)
                    atomicOr(count + at, 0x80000000u);
                else
                    atomicAdd(count + at, 1u);
            };
            const int head = min(len, (int)(-(reinterpret_cast<intptr_t>(h) / 4) & 3)), quads = (len - head) / 4;
            if (tid < head) add(h[tid], tid);
#pragma unroll 4
            for (int i = tid; i < quads; i += LOGITS_THREADS) {
                const int4 w = reinterpret_cast<const int4 *>(h + head)[i];
                const int at = head + 4 * i;
                add(w.x, at), add(w.y, at + 1), add(w.z, at + 2), add(w.w, at + 3);
            }
            const int tail = head + 4 * quads + tid;
            if (tail < len) add(h[tail], tail);
            for (int i = tid; i < entries; i += LOGITS_THREADS) {
                const int at = place(a.how.bias_ids[start + i]);
                if ((unsigned)at < (unsigned)n) atomicMax(entry + at, (uint32_t)i + 1u);
            }
        }
        auto path = [&](uint32_t by) {  // the row's drafts
            if (!known || !a.how.drafts) return;
            const int first = min(max(a.how.q_start[s], 0), a.rows), drafts = min(max(a.how.q_start[s + 1], 0), a.rows) - first;
            const int bits = (int)min((int64_t)drafts, (int64_t)32 * a.how.words);
            const uint32_t *tree = a.how.tree + (int64_t)row * a.how.words;
            for (int i = tid; i < bits; i += LOGITS_THREADS)
                if (tree[i >> 5] >> (i & 31) & 1) {
                    const int at = place(a.how.drafts[first + i]);
                    if ((unsigned)at < (unsigned)n) atomicAdd(count + at, by);
                }
        };
        path(1u);
        __syncthreads();

        auto adjust = [&](float y, uint32_t c, uint32_t e) {
            if (e) y += bias[e - 1];
            if (c) {
                y = y > 0.0f ? __fdiv_rn(y, rep) : y * rep;
                const uint32_t times = c & 0x7fffffffu;
                if (times) y = fmaf(-freq, (float)times, y) - pres;
            }
            return y;
        };
#pragma unroll
        for (int u = 0; u < LOGITS_U; ++u) {
            const int q = tid + u * LOGITS_THREADS, at = 4 * q, id = ids0 + at;
            if (at >= n) break;
            const uint4 c = reinterpret_cast<const uint4 *>(count)[q];
            const uint4 e = a.has_bias ? reinterpret_cast<const uint4 *>(entry)[q] : make_uint4(0, 0, 0, 0);
            const uint32_t ok = a.how.allow ? mask[at >> 5] >> (at & 31) & 15u : 15u;
            const bool touched = (c.x | c.y | c.z | c.w | e.x | e.y | e.z | e.w) != 0;
            if (in_place) {
                if (ok == 15u && !touched) continue;
                if (ok != 0u || !whole(q)) fetch(v[u], q);
            }
            float y[4];
            v[u].get(y);
            if (touched) {
                y[0] = adjust(y[0], c.x, e.x), y[1] = adjust(y[1], c.y, e.y);
                y[2] = adjust(y[2], c.z, e.z), y[3] = adjust(y[3], c.w, e.w);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = ok >> k & 1 ? y[k] : -INFINITY;
            if (whole(q)) {
                store_vec<O, 4>(out + id, y);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (id + k >= 0 && at + k < n) out[id + k] = from_f32<O>(y[k]);
            }
        }
        if (row + 1 < row1) {
            __syncthreads();
            path(0xffffffffu);  // off again
            if (a.how.drafts) __syncthreads();
        }
    }
}

// Segments of a row, and whether they and the rows are counted in 32 bits.
static int64_t logits_segments(int V, int seg) { return ((int64_t)V + 3 + seg - 1) / seg; }

template <class I, class O>
static int logits_launch(const LogitsArgs &a, cudaStream_t s) {
    const uint32_t bytes = (uint32_t)a.seg * (a.has_bias ? 8 : 4) + a.seg / 8;
    const int64_t groups = (a.rows + (int64_t)a.group - 1) / a.group;
    return launch_programmatic(logits_kernel<I, O>, dim3((unsigned)(groups * logits_segments(a.V, a.seg))), LOGITS_THREADS, bytes, s, a) ? QG_OK
                                                                                                                                       : QG_ECUDA;
}
template <class I>
static int logits_out(const LogitsArgs &a, int out_type, cudaStream_t s) {
    switch (out_type) {
    case QG_F32: return logits_launch<I, float>(a, s);
    case QG_F16: return logits_launch<I, f16>(a, s);
    default: return logits_launch<I, bf16>(a, s);
    }
}

}  // namespace qg

using namespace qg;

extern "C" {

int qg_tree_masks(const int32_t *parents, const int32_t *q_start, const int32_t *kv_len, int tokens, int batch, uint32_t *tree, int words,
                  int32_t *positions, void *stream) {
    if (!parents || !q_start || !kv_len || !tree || !positions || tokens < 1 || batch < 1 || words < 1 || words > TREE_MAX / 32 || batch == INT32_MAX)
        return QG_EINVAL;
    for (const void *p : {(const void *)parents, (const void *)q_start, (const void *)kv_len, (const void *)tree, (const void *)positions})
        if (!host_aligned(p, 4)) return QG_EALIGN;
    const int sms = device_sms();
    if (sms < 0) return sms;
    return launch_programmatic(tree_masks_kernel, dim3((unsigned)batch + 1), TREE_THREADS, 0, (cudaStream_t)stream, parents, q_start, kv_len,
                               tokens, batch, tree, words, positions)
               ? QG_OK
               : QG_ECUDA;
}

int qg_cache_keep(const int32_t *keep, int64_t keep_stride, const int32_t *keep_len, int width, int layers, int64_t layer_stride,
                  int64_t step_layer_stride, int32_t *kv_out, const qg_paged *cache, void *stream) {
    if (!keep || !keep_len || !kv_out || !cache || width < 1 || width > KEEP_MAX || keep_stride < width || layers < 1 || layers > 65535)
        return QG_EINVAL;
    if (const int rc = paged_check(*cache)) return rc;
    const bool q8 = cache->type == QG_Q8_0;
    const int es = q8 ? 1 : 2;
    if (cache->batch > 65535 || (layers > 1 && (layer_stride < 1 || (q8 && step_layer_stride < 1)))) return QG_EINVAL;
    if (!host_aligned(keep, 4) || !host_aligned(keep_len, 4) || !host_aligned(kv_out, 4)) return QG_EALIGN;
    if (layers > 1 && (layer_stride * es % 16 || (q8 && step_layer_stride % 8))) return QG_EALIGN;
    KeepArgs a{};
    a.heads = cache->kv_heads;
    a.chunks = cache->dim * es / 16;
    a.step_words = q8 ? cache->dim / 64 : 0;
    const int64_t items = 2 * (int64_t)a.heads * (a.chunks + a.step_words);
    if (items > INT32_MAX - KEEP_THREADS) return QG_EINVAL;
    const int sms = device_sms();
    if (sms < 0) return sms;
    a.bt = paged_batch(*cache, INT32_MAX);  // no array of tokens is touched
    a.keep = keep, a.keep_len = keep_len, a.keep_stride = keep_stride, a.width = width;
    const bool over = kv_out == cache->kv_len;
    a.kv_out = over ? nullptr : kv_out;
    a.k = static_cast<uint8_t *>(cache->k), a.v = static_cast<uint8_t *>(cache->v);
    a.kd = static_cast<uint8_t *>(cache->kd), a.vd = static_cast<uint8_t *>(cache->vd);
    a.layer = layer_stride * es, a.page_stride = cache->page_stride * es;
    a.head_stride = cache->head_stride * es, a.slot_stride = cache->slot_stride * es;
    a.step_layer = step_layer_stride * 2, a.step_page = cache->step_stride * 2;
    cudaStream_t s = (cudaStream_t)stream;
    const dim3 grid((unsigned)((items + KEEP_THREADS - 1) / KEEP_THREADS), (unsigned)cache->batch, (unsigned)layers);
    if (!launch_programmatic(cache_keep_kernel, grid, KEEP_THREADS, 0, s, a)) return QG_ECUDA;
    if (!over) return QG_OK;
    return launch_programmatic(keep_lengths_kernel, dim3(((unsigned)cache->batch + KEEP_THREADS - 1) / KEEP_THREADS), KEEP_THREADS, 0, s, a, kv_out)
               ? QG_OK
               : QG_ECUDA;
}

int qg_logits_adjust(const void *logits, int type, int64_t ld, void *out, int out_type, int64_t ldo, int rows, int V, const qg_logits *how,
                     void *stream) {
    if (!logits || !out || !how || !float_type(type) || !float_type(out_type) || rows < 1 || V < 1 || V > INT32_MAX - 2 * LOGITS_SEG || ld < V ||
        ldo < V)
        return QG_EINVAL;
    const qg_logits &h = *how;
    const bool sequences = h.history || h.drafts || h.repetition || h.frequency || h.presence || h.bias_start;
    if (h.batch < 0 || (sequences && h.batch < 1) || (h.history && (!h.history_len || h.history_stride < 0 || h.history_width < 0))) return QG_EINVAL;
    if ((h.drafts || h.tree) && (!h.drafts || !h.tree || !h.q_start || h.words < 1)) return QG_EINVAL;
    if (h.bias_start && (!h.bias_ids || !h.bias || h.bias_entries < 0)) return QG_EINVAL;
    if (h.allow && h.allow_stride < (V + 31) / 32) return QG_EINVAL;
    if (out == logits && (type != out_type || ld != ldo)) return QG_EINVAL;
    if (!host_aligned(logits, type_size(type)) || !host_aligned(out, type_size(out_type))) return QG_EALIGN;
    for (const void *p : {(const void *)h.seq, (const void *)h.history, (const void *)h.history_len, (const void *)h.prompt_len,
                          (const void *)h.repetition, (const void *)h.frequency, (const void *)h.presence, (const void *)h.bias_start,
                          (const void *)h.bias_ids, (const void *)h.bias, (const void *)h.allow, (const void *)h.drafts, (const void *)h.tree,
                          (const void *)h.q_start})
        if (!host_aligned(p, 4)) return QG_EALIGN;
    LogitsArgs a{logits, out, ld, ldo, V, 0, rows, 1, out == logits, h.bias_start != nullptr, h};
    const int64_t fill = 4 * (int64_t)device_sms_planning();  // blocks that run at once
    a.seg = (int)std::min<int64_t>(std::max<int64_t>(rows * (int64_t)V / fill / 128 * 128 + 128, 512), LOGITS_SEG);
    // rows that may share a sequence share a block, as long as every SM has a few blocks to overlap
    if (h.seq && sequences) a.group = (int)std::min<int64_t>(std::max<int64_t>(rows * logits_segments(V, a.seg) / (2 * fill), 1), 8);
    if (rows * logits_segments(V, a.seg) > INT32_MAX) return QG_EINVAL;
    const int sms = device_sms();
    if (sms < 0) return sms;
    cudaStream_t s = (cudaStream_t)stream;
    switch (type) {
    case QG_F32: return logits_out<float>(a, out_type, s);
    case QG_F16: return logits_out<f16>(a, out_type, s);
    default: return logits_out<bf16>(a, out_type, s);
    }
}

}  // extern "C"
