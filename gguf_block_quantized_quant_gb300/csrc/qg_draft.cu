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
// indices, pages, data); the bytes that move are few: 5 of 16 drafts in one layer of 8 heads of 128 2.6 us in a graph (4 to 5 called
// one by one), 6 of 48 in 32 sequences and 16 layers 5.5 us, of which the bytes are 2.8.
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
// What changes most logits, the mask, and what changes a few, biases and penalties, are apart: the logits stream past the
// mask, then the ids that have a bias or were said go over that.  For these a block takes a segment of ids for a few rows.  For each
// sequence among them it counts the ids of the segment that the history holds in shared memory (a word per id), notes
// the last bias entry of each, and lists the ids so touched; the drafts that each row follows, few or none of which fall into a
// segment, are listed per row.  Whole numbers are added, so the order of the atomics changes nothing but the lists'.
// The stream is bound by memory, the rest by a chain of dependent loads (sequence, lengths, ids, logits).  Small calls do both in
// one kernel; large ones stream in a kernel of many light blocks, under whose end the counts of a second are made.  One
// kernel for 192 rows of 131071, bf16 to fp32: 97 us with the counts beside the stream, 60 to 70 with lists, as the chains
// of the few blocks that fit an SM do not hide each other; two kernels 48 us, of which the stream is 28 (0.83 of the
// measured copy bandwidth).  One row of 32000, fp32, a history of 600: 4.2 us.
struct LogitsArgs {
    const void *x;
    void *out;
    int64_t ld, ldo;  // elements
    int V, seg;       // seg: ids of a segment at most, a multiple of 8
    int shift;        // a segment holds every 2^shift-th id, as often said ones are near each other; 0: neighbouring ids, to stream them
    int rows, group;  // group: rows of a block
    int in_place, stream, counts, has_bias;  // stream: the logits go past the mask here too; counts: some row has a history, drafts or biases
    qg_logits how;
};

// Segments of a row.
__host__ __device__ constexpr int logits_segments(int V, int seg, int shift = 0) { return shift ? 1 << shift : (int)(((int64_t)V + seg - 1) / seg); }

constexpr int LOGITS_HISTORY = 1 << 29;  // ids of a history that count; with the drafts below TIMES
constexpr int LOGITS_THREADS = 256, LOGITS_U = 4, LOGITS_SEG = 4096, LOGITS_GROUP = 16;
constexpr int LOGITS_PATH = 30;          // drafts of a row in a segment that are listed; where there are more, all are looked through

// A word of the counts: how often the id was said after the prompt, that it was said before, that it has a bias.  No id
// whose word is 0 is listed.
constexpr uint32_t SAID = 0x80000000u, BIASED = 0x40000000u, TIMES = 0x3fffffffu;

// Four elements as they come, read once: the second-level cache is for the output.
template <class T>
struct Raw4 {
    uint2 w;
    __device__ __forceinline__ void load(const T *p) { w = __ldcs(reinterpret_cast<const uint2 *>(p)); }
    __device__ __forceinline__ void get(float (&v)[4]) const {
        const float2 a = unpack2<T>(w.x), b = unpack2<T>(w.y);
        v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    }
};
template <>
struct Raw4<float> {
    float4 w;
    __device__ __forceinline__ void load(const float *p) { w = __ldcs(reinterpret_cast<const float4 *>(p)); }
    __device__ __forceinline__ void get(float (&v)[4]) const { v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w; }
};

// The row's bit of id v, and four from it on (v + 3 < V).
__device__ __forceinline__ uint32_t allowed(const uint32_t *row, int v) { return row[v >> 5] >> (v & 31) & 1u; }
__device__ __forceinline__ uint32_t allowed4(const uint32_t *row, int v) { return __funnelshift_r(row[v >> 5], row[(v + 3) >> 5], v & 31) & 15u; }

// Ids id0 .. id1 - 1 of a row, past the mask.
template <class I, class O>
__device__ __forceinline__ void logits_stream(const LogitsArgs &a, int row, int id0, int id1) {
    const int tid = LOGITS_THREADS - 1 - threadIdx.x;  // the first warps have the ids of a short history to count
    const I *x = static_cast<const I *>(a.x) + row * a.ld;
    O *out = static_cast<O *>(a.out) + row * a.ldo;
    const uint32_t *allow = a.how.allow ? a.how.allow + row * a.how.allow_stride : nullptr;
    const bool in_place = std::is_same<I, O>::value && a.in_place;
    if (in_place && !allow) return;
    auto one = [&](int v) {
        const bool ok = !allow || allowed(allow, v);
        if (!(in_place && ok)) out[v] = ok ? from_f32<O>(to_f32(x[v])) : from_f32<O>(-INFINITY);
    };
    // vectors start where four elements of `out` do; x has to be at the same place between its own boundaries
    const int lead = (int)((reinterpret_cast<uintptr_t>(out + id0) / sizeof(O)) & 3);
    if ((int)((reinterpret_cast<uintptr_t>(x + id0) / sizeof(I)) & 3) != lead) {
        for (int v = id0 + tid; v < id1; v += LOGITS_THREADS) one(v);
        return;
    }
    const int head = min((4 - lead) & 3, id1 - id0), quads = (id1 - id0 - head) / 4, v0 = id0 + head, left = id1 - v0 - 4 * quads;
    if (tid < head) one(id0 + tid);
    if (tid < left) one(id1 - left + tid);
    for (int q0 = tid; q0 < quads; q0 += LOGITS_THREADS * LOGITS_U) {
        Raw4<I> r[LOGITS_U];
        uint32_t ok[LOGITS_U];
#pragma unroll
        for (int u = 0; u < LOGITS_U; ++u) {
            const int q = q0 + u * LOGITS_THREADS, v = v0 + 4 * q;
            if (q >= quads) continue;
            ok[u] = allow ? allowed4(allow, v) : 15u;
            if (!in_place || (ok[u] != 0u && ok[u] != 15u)) r[u].load(x + v);
        }
#pragma unroll
        for (int u = 0; u < LOGITS_U; ++u) {
            const int q = q0 + u * LOGITS_THREADS;
            if (q >= quads || (in_place && ok[u] == 15u)) continue;
            float y[4];
            r[u].get(y);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = ok[u] >> k & 1 ? y[k] : -INFINITY;
            store_vec<O, 4>(out + v0 + 4 * q, y);
        }
    }
}

template <class I, class O>
__global__ void __launch_bounds__(LOGITS_THREADS, 4) logits_kernel(const __grid_constant__ LogitsArgs a) {
    extern __shared__ __align__(16) uint32_t lg_smem[];
    __shared__ int touched, seqs[LOGITS_GROUP], paths[LOGITS_GROUP];
    __shared__ uint16_t path[LOGITS_GROUP][LOGITS_PATH];
    uint32_t *count = lg_smem;
    uint32_t *entry = count + a.seg;                                                       // where there are biases
    uint16_t *list = reinterpret_cast<uint16_t *>(entry + (a.has_bias ? a.seg : 0));
    const int tid = threadIdx.x;
    const int segs = logits_segments(a.V, a.seg, a.shift);
    const int row0 = (int)(blockIdx.x / segs) * a.group, rows = min(a.group, a.rows - row0);
    const int seg = (int)(blockIdx.x % segs), id0 = a.shift ? seg : seg * a.seg, id1 = a.shift ? a.V : min(id0 + a.seg, a.V);
    const int n = (int)(((int64_t)id1 - id0 + (1 << a.shift) - 1) >> a.shift);
    // the place of an id in the segment, from n on for others; ids below 0 are far away
    auto place = [&](int id) {
        const unsigned d = (unsigned)id - (unsigned)id0;
        return d & ((1u << a.shift) - 1u) ? 0xffffffffu : d >> a.shift;
    };
    // After a stream kernel nothing that it writes is read yet, and what that waited for is complete; the ids are read past
    // the first-level cache, which may hold what was there before
    if (a.stream) griddep_wait();
    if (tid < rows) {
        const int s = a.how.seq ? __ldcg(a.how.seq + row0 + tid) : row0 + tid;
        seqs[tid] = (unsigned)s < (unsigned)a.how.batch ? s : -1;
    }
    if (a.counts)
        for (int i = tid; i < a.seg / 4; i += LOGITS_THREADS) reinterpret_cast<uint4 *>(count)[i] = make_uint4(0, 0, 0, 0);
    if (a.has_bias)
        for (int i = tid; i < a.seg / 4; i += LOGITS_THREADS) reinterpret_cast<uint4 *>(entry)[i] = make_uint4(0, 0, 0, 0);
    if (tid < LOGITS_GROUP) paths[tid] = 0;
    if (tid == 0) touched = 0;
    __syncthreads();

    for (int r0 = 0, r1; r0 < rows; r0 = r1) {  // rows r0 .. r1 - 1 of the block belong to sequence s
        const int s = seqs[r0];
        for (r1 = r0 + 1; r1 < rows && seqs[r1] == s; ++r1) {}
        auto listed = [&](int at, uint32_t before) {
            if (before == 0) list[atomicAdd(&touched, 1)] = (uint16_t)at;
        };
        const float *bias = nullptr;
        float rep = 1.0f, freq = 0.0f, pres = 0.0f;
        int first = 0, bits = 0;  // of the sequence's drafts
        if (s >= 0) {
            if (a.how.repetition) rep = __ldcg(a.how.repetition + s);
            if (a.how.frequency) freq = __ldcg(a.how.frequency + s);
            if (a.how.presence) pres = __ldcg(a.how.presence + s);
            if (a.how.drafts) {
                first = min(max(__ldcg(a.how.q_start + s), 0), a.rows);
                bits = (int)min((int64_t)(min(max(__ldcg(a.how.q_start + s + 1), 0), a.rows) - first), (int64_t)32 * a.how.words);
            }
            int start = 0, entries = 0;
            if (a.has_bias) {
                start = min(max(__ldcg(a.how.bias_start + s), 0), a.how.bias_entries);
                entries = min(__ldcg(a.how.bias_start + s + 1), a.how.bias_entries) - start;
                bias = a.how.bias + start;
            }
            if (a.how.history) {
                const int len = min(max(__ldcg(a.how.history_len + s), 0), min(a.how.history_width, LOGITS_HISTORY));
                const int said = a.how.prompt_len ? __ldcg(a.how.prompt_len + s) : 0;
                const int32_t *h = a.how.history + s * a.how.history_stride;
                auto add = [&](int id, int i) {
                    const unsigned at = place(id);
                    if (at < (unsigned)n) listed((int)at, i < said ? atomicOr(count + at, SAID) : atomicAdd(count + at, 1u));
                };
                const int head = min(len, (int)(-(reinterpret_cast<intptr_t>(h) / 4) & 3)), quads = (len - head) / 4;
                if (tid < head) add(__ldcg(h + tid), tid);
#pragma unroll 4
                for (int i = tid; i < quads; i += LOGITS_THREADS) {
                    const int4 w = __ldcg(reinterpret_cast<const int4 *>(h + head) + i);
                    const int at = head + 4 * i;
                    add(w.x, at), add(w.y, at + 1), add(w.z, at + 2), add(w.w, at + 3);
                }
                const int tail = head + 4 * quads + tid;
                if (tail < len) add(__ldcg(h + tail), tail);
            }
            for (int i = tid; i < entries; i += LOGITS_THREADS) {
                const unsigned at = place(__ldcg(a.how.bias_ids + start + i));
                if (at >= (unsigned)n) continue;
                listed((int)at, atomicOr(count + at, BIASED));
                atomicMax(entry + at, (uint32_t)i + 1u);
            }
        }
        // the drafts that row r0 + r of the block follows: bit i, its place in the segment (or beyond it)
        auto follows = [&](int r, int i) { return __ldcg(a.how.tree + (int64_t)(row0 + r) * a.how.words + (i >> 5)) >> (i & 31) & 1u; };
        auto draft = [&](int i) { return place(__ldcg(a.how.drafts + first + i)); };
        for (int64_t x = tid; x < (int64_t)(r1 - r0) * bits; x += LOGITS_THREADS) {
            const int r = r0 + (int)(x / bits), i = (int)(x % bits);
            const unsigned at = draft(i);
            if (follows(r, i) && at < (unsigned)n) {
                const int k = atomicAdd(&paths[r], 1);
                if (k < LOGITS_PATH) path[r][k] = (uint16_t)at;
            }
        }
        if (r0 == 0) {
            if (a.stream) {
                griddep_launch_dependents();
                for (int r = 0; r < rows; ++r) logits_stream<I, O>(a, row0 + r, id0, id1);
            } else {
                griddep_wait();
                griddep_launch_dependents();
            }
        }
        __syncthreads();  // what is listed goes over what the stream wrote

        // Ids with the words c that the row's drafts leave them: loads of several are in flight together.  What the stream wrote is
        // the logit itself, masked, and nearer by than that, but where the output is narrower; -inf stays what it is
        constexpr int MANY = 4;
        constexpr bool WRITTEN = std::is_same<I, O>::value || std::is_same<O, float>::value;
        auto put = [&](const int (&r)[MANY], const unsigned (&at)[MANY], const uint32_t (&c)[MANY], int have) {
            float y[MANY];
            bool ok[MANY];
#pragma unroll
            for (int u = 0; u < MANY; ++u) {
                const int row = row0 + r[u], id = id0 + (int)(at[u] << a.shift);
                ok[u] = u < have;
                if (!ok[u]) continue;
                if constexpr (WRITTEN) {
                    y[u] = to_f32(static_cast<const O *>(a.out)[row * a.ldo + id]);
                } else {
                    y[u] = to_f32(static_cast<const I *>(a.x)[row * a.ld + id]);
                    if (a.how.allow) ok[u] = allowed(a.how.allow + row * a.how.allow_stride, id);
                }
            }
#pragma unroll
            for (int u = 0; u < MANY; ++u) {
                if (!ok[u] || y[u] == -INFINITY) continue;
                if (c[u] & BIASED) y[u] += bias[entry[at[u]] - 1];
                if (c[u] & ~BIASED) y[u] = y[u] > 0.0f ? __fdiv_rn(y[u], rep) : y[u] * rep;
                if (c[u] & TIMES) y[u] = fmaf(-freq, (float)(c[u] & TIMES), y[u]) - pres;
                static_cast<O *>(a.out)[(row0 + r[u]) * a.ldo + id0 + (int)(at[u] << a.shift)] = from_f32<O>(y[u]);
            }
        };
        auto times = [&](int r, unsigned at) {  // how often the row's drafts say the id
            uint32_t k = 0;
            if (paths[r] <= LOGITS_PATH) {
                for (int i = 0; i < paths[r]; ++i) k += path[r][i] == at;
            } else {
                for (int i = 0; i < bits; ++i) k += follows(r, i) && draft(i) == at;
            }
            return k;
        };
        const int ids = touched;
        for (int x = tid; x < (r1 - r0) * ids; x += LOGITS_THREADS * MANY) {
            int r[MANY], have = 0;
            unsigned at[MANY];
            uint32_t c[MANY];
#pragma unroll
            for (int u = 0; u < MANY; ++u) {
                const int y = x + u * LOGITS_THREADS;
                if (y >= (r1 - r0) * ids) break;
                r[u] = r0 + y / ids;
                at[u] = list[y % ids];
                c[u] = count[at[u]] + times(r[u], at[u]);
                have = u + 1;
            }
            put(r, at, c, have);
        }
        // ids that a row's drafts alone say: each once, at its first place among them
        auto one = [&](int r, unsigned at) {
            const int rs[MANY] = {r};
            const unsigned ats[MANY] = {at};
            const uint32_t cs[MANY] = {times(r, at)};
            put(rs, ats, cs, 1);
        };
        if (bits > 0) {
            for (int x = tid; x < (r1 - r0) * LOGITS_PATH; x += LOGITS_THREADS) {
                const int r = r0 + x / LOGITS_PATH, k = x % LOGITS_PATH;
                if (paths[r] > LOGITS_PATH || k >= paths[r] || count[path[r][k]] != 0) continue;
                bool again = false;
                for (int i = 0; i < k; ++i) again = again || path[r][i] == path[r][k];
                if (!again) one(r, path[r][k]);
            }
            for (int r = r0; r < r1; ++r) {  // rows with more than the list holds
                if (paths[r] <= LOGITS_PATH) continue;
                for (int i = tid; i < bits; i += LOGITS_THREADS) {
                    const unsigned at = draft(i);
                    if (at >= (unsigned)n || count[at] != 0 || !follows(r, i)) continue;
                    bool again = false;
                    for (int k = 0; k < i && !again; ++k) again = follows(r, k) && draft(k) == at;
                    if (!again) one(r, at);
                }
            }
        }
        if (r1 < rows) {  // another sequence
            __syncthreads();
            for (int i = tid; i < ids; i += LOGITS_THREADS) {
                count[list[i]] = 0u;
                if (a.has_bias) entry[list[i]] = 0u;
            }
            if (tid == 0) touched = 0;
            __syncthreads();
        }
    }
}

template <class I, class O>
__global__ void __launch_bounds__(LOGITS_THREADS, 8) logits_stream_kernel(const __grid_constant__ LogitsArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    const int segs = (a.V + LOGITS_SEG - 1) / LOGITS_SEG;
    const int64_t total = (int64_t)a.rows * segs;
    for (int64_t i = blockIdx.x; i < total; i += gridDim.x) {
        const int id0 = (int)(i % segs) * LOGITS_SEG;
        logits_stream<I, O>(a, (int)(i / segs), id0, min(id0 + LOGITS_SEG, a.V));
    }
}

template <class I, class O>
static int logits_launch(LogitsArgs a, int sms, cudaStream_t s) {
    if (!a.stream && !(a.in_place && !a.how.allow)) {
        const int64_t blocks = std::min<int64_t>((int64_t)a.rows * logits_segments(a.V, LOGITS_SEG), 8 * (int64_t)sms);
        if (!launch_programmatic(logits_stream_kernel<I, O>, dim3((unsigned)blocks), LOGITS_THREADS, 0, s, a)) return QG_ECUDA;
        if (!a.counts) return QG_OK;
    } else if (!a.stream) {
        a.stream = 1;  // nothing streams, but the kernel is the call's first
    }
    const uint32_t bytes = (uint32_t)a.seg * (a.has_bias ? 10 : 6);
    const int64_t groups = (a.rows + (int64_t)a.group - 1) / a.group;
    return launch_programmatic(logits_kernel<I, O>, dim3((unsigned)(groups * logits_segments(a.V, a.seg, a.shift))), LOGITS_THREADS, bytes, s, a) ? QG_OK
                                                                                                                                       : QG_ECUDA;
}
template <class I>
static int logits_out(const LogitsArgs &a, int out_type, int sms, cudaStream_t s) {
    switch (out_type) {
    case QG_F32: return logits_launch<I, float>(a, sms, s);
    case QG_F16: return logits_launch<I, f16>(a, sms, s);
    default: return logits_launch<I, bf16>(a, sms, s);
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
    const int64_t fill = 4 * (int64_t)device_sms_planning();  // blocks of the kernel with the counts that run at once
    const bool counts = h.history || h.drafts || h.bias_start;
    LogitsArgs a{logits, out, ld, ldo, V, 0, 0, rows, 1, out == logits, 1, counts, h.bias_start != nullptr, h};
    a.seg = (int)std::min<int64_t>(std::max<int64_t>(rows * (int64_t)V / fill / 128 * 128 + 128, 512), LOGITS_SEG);
    // One kernel up to where its blocks run at once, else as many rows for each block of the second as let them
    a.stream = (int64_t)rows * logits_segments(V, a.seg) <= fill;
    if (!a.stream) {
        for (a.seg = LOGITS_SEG; (int64_t)a.seg << a.shift < V; ++a.shift) {}
        a.group = (int)std::min<int64_t>((((int64_t)rows << a.shift) + fill - 1) / fill, LOGITS_GROUP);
        // rows that divide evenly over the sequences are taken for runs of as many: a block takes whole ones
        const int run = h.seq && h.batch > 0 && rows % h.batch == 0 ? rows / h.batch : 1;
        if (run <= LOGITS_GROUP) a.group = std::min((a.group + run - 1) / run, LOGITS_GROUP / run) * run;
    }
    if ((int64_t)rows * logits_segments(V, a.seg, a.shift) > INT32_MAX) return QG_EINVAL;
    const int sms = device_sms();
    if (sms < 0) return sms;
    cudaStream_t s = (cudaStream_t)stream;
    switch (type) {
    case QG_F32: return logits_out<float>(a, out_type, sms, s);
    case QG_F16: return logits_out<f16>(a, out_type, sms, s);
    default: return logits_out<bf16>(a, out_type, sms, s);
    }
}

}  // extern "C"
