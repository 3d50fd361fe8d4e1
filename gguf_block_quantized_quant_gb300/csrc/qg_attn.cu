// qg_attn.cu -- attention over a paged cache: the C entry points and tensor maps.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <mutex>
#include <set>
#include <utility>

#include "qg_attn.cuh"
#include "qg_launch.h"

namespace qg {

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

int attn_dev_err_take(unsigned int *err) {
    unsigned int v[6] = {};
    *err = 0;
    for (const int rc : {attn_rows_dev_err_take<MOD_PLAIN>(&v[0]), attn_chunk_dev_err_take<MOD_PLAIN>(&v[1]),
                         attn_rows_dev_err_take<MOD_SHAPED>(&v[2]), attn_chunk_dev_err_take<MOD_SHAPED>(&v[3]),
                         attn_chunk_dev_err_take<MOD_CAPPED>(&v[4]), attn_chunk_dev_err_take<MOD_BIASED>(&v[5])})
        if (rc) return rc;
    for (const unsigned int x : v) *err |= x;
    return QG_OK;
}

// The arguments that every attention call has, checked, and the kernels' view of them.
static int attn_args(AttnArgs &a, const void *q, int64_t ldq, int64_t hdq, int q_type, int tokens, int q_heads, int max_new, float scale,
                     int window, void *out, int out_type, float *lse, const qg_paged *cache, void *ws, size_t ws_bytes, int &sms) {
    if (!q || !out || !cache || tokens < 1 || q_heads < 1 || max_new < 0 || window < 0 || !(scale == scale)) return QG_EINVAL;
    if (const int rc = paged_check(*cache)) return rc;
    if (q_type != (cache->type == QG_BF16 ? QG_BF16 : QG_F16) || (out_type != q_type && out_type != QG_F32)) return QG_EINVAL;
    const int D = cache->dim;
    if (q_heads % cache->kv_heads || ldq < D || hdq < D) return QG_EINVAL;
    if ((int64_t)tokens * q_heads > INT32_MAX) return QG_EINVAL;  // rows of out are counted in 32 bits
    if (!host_aligned(q, 16) || ldq % 8 || hdq % 8 || !host_aligned(out, 16) || !host_aligned(lse, 4)) return QG_EALIGN;
    if (!ws || ws_bytes < qg_attn_workspace_size(D, q_heads, cache->kv_heads, tokens, cache->batch)) return QG_EWORKSPACE;
    if (!host_aligned(ws, 16)) return QG_EALIGN;
    sms = device_sms();
    if (sms < 0) return sms;
    a = AttnArgs{};
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
    return QG_OK;
}

// One row tile of 16 per sequence and cache head: the row kernel reads the cache once.  Else the chunk kernel.
static int attn_plain(const AttnArgs &a, const qg_paged &c, int max_new, int sms, cudaStream_t s) {
    if ((int64_t)max_new * a.G > DEC_ROWS) return attn_chunk<MOD_PLAIN>(a, c, sms, s);
    return attn_rows<MOD_PLAIN>(a, c, (int64_t)max_new * a.G <= 8 ? 1 : 2, sms, s);
}
// With several row tiles per sequence and cache head the row kernel reads the cache as often, but spares the plan and some
// microseconds of the chunk kernel's start: that wins where the tiles are few and the caches, as large as the page table
// allows, small.  us, chunk and row kernel (fp16, 32/8 heads of 128): 16 drafts of one sequence after 1000 18.6, 15.8; 8
// after 4000 22.1, 17.5; 32 after 1000 20.9, 22.2; 8 of 4 sequences after 1000 22.0, 20.9; 16 after 300 20.2, 21.7.  (16-bit
// heads of 256: 8 after 1000 18.5, 19.8.)  The host knows no lengths but the table's: one as wide as the longest sequence that a
// server allows sends a small tree to the chunk kernel whatever its length.
static bool few_rows(const AttnArgs &a, const qg_paged &c, int max_new) {
    const int64_t rows = (int64_t)max_new * a.G;
    if (rows <= DEC_ROWS) return true;
    const int64_t tiles = (rows + DEC_ROWS - 1) / DEC_ROWS;
    if (tiles * c.batch * a.Hk > 64 || (c.dim == 256 && c.type != QG_Q8_0)) return false;
    const int64_t slot = 2 * (int64_t)a.Hk * (c.type == QG_Q8_0 ? c.dim + c.dim / 16 : c.dim * 2);
    return (tiles - 1) * c.batch * std::min<int64_t>((int64_t)c.table_width * c.page, MAX_SLOTS) <= (int64_t)(16 << 20) / slot;
}
static int attn_other(const AttnArgs &a, const qg_paged &c, int max_new, int sms, cudaStream_t s) {
    if (!few_rows(a, c, max_new))
        return a.sh.slopes            ? attn_chunk<MOD_BIASED>(a, c, sms, s)
               : a.sh.cap_out > 0.0f ? attn_chunk<MOD_CAPPED>(a, c, sms, s)
                                     : attn_chunk<MOD_SHAPED>(a, c, sms, s);
    return attn_rows<MOD_SHAPED>(a, c, (int64_t)max_new * a.G <= 8 ? 1 : 2, sms, s);
}

// The cap and the slopes of a call.  A quotient scale / cap below the normal numbers has lost the bits of the scale.
static int shape_check(float scale, float cap, const float *slopes) {
    if (!(cap >= 0.0f)) return QG_EINVAL;
    if (cap > 0.0f && (!std::isfinite(scale / cap) || !std::isfinite(cap * LOG2E) || (scale != 0.0f && std::abs(scale / cap) < FLT_MIN))) return QG_EINVAL;
    return host_aligned(slopes, 4) ? QG_OK : QG_EALIGN;
}
static void shape_scores(AttnArgs &a, float scale, float cap, const float *slopes) {
    if (cap > 0.0f) a.sh.cap_in = scale / cap, a.sh.cap_out = cap * LOG2E;
    a.sh.slopes = slopes;
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
    AttnArgs a;
    int sms;
    if (const int rc = attn_args(a, q, ldq, hdq, q_type, tokens, q_heads, max_new, scale, window, out, out_type, lse, cache, ws, ws_bytes, sms))
        return rc;
    return attn_plain(a, *cache, max_new, sms, (cudaStream_t)stream);
}

int qg_attn_shaped(const void *q, int64_t ldq, int64_t hdq, int q_type, int tokens, int q_heads, int max_new, float scale, int window,
                   float cap, const float *slopes, const int32_t *prefix, const int32_t *first, void *out, int out_type, float *lse,
                   const qg_paged *cache, void *ws, size_t ws_bytes, void *stream) {
    if (const int rc = shape_check(scale, cap, slopes)) return rc;
    if (!host_aligned(prefix, 4) || !host_aligned(first, 4)) return QG_EALIGN;
    AttnArgs a;
    int sms;
    if (const int rc = attn_args(a, q, ldq, hdq, q_type, tokens, q_heads, max_new, scale, window, out, out_type, lse, cache, ws, ws_bytes, sms))
        return rc;
    shape_scores(a, scale, cap, slopes);
    a.sh.prefix = prefix, a.sh.first = first;
    // nothing that the plain kernels do not do
    if (!(cap > 0.0f) && !slopes && !prefix && !first) return attn_plain(a, *cache, max_new, sms, (cudaStream_t)stream);
    return attn_other(a, *cache, max_new, sms, (cudaStream_t)stream);
}

int qg_attn_tree(const void *q, int64_t ldq, int64_t hdq, int q_type, int tokens, int q_heads, int max_new, float scale, int window,
                 float cap, const float *slopes, const uint32_t *tree, int words, const int32_t *positions, void *out, int out_type,
                 float *lse, const qg_paged *cache, void *ws, size_t ws_bytes, void *stream) {
    if (!tree || words < 1) return QG_EINVAL;
    if (const int rc = shape_check(scale, cap, slopes)) return rc;
    if (!host_aligned(tree, 4) || !host_aligned(positions, 4)) return QG_EALIGN;
    AttnArgs a;
    int sms;
    if (const int rc = attn_args(a, q, ldq, hdq, q_type, tokens, q_heads, max_new, scale, window, out, out_type, lse, cache, ws, ws_bytes, sms))
        return rc;
    shape_scores(a, scale, cap, slopes);
    a.sh.tree = tree, a.sh.words = words, a.sh.positions = positions;
    return attn_other(a, *cache, max_new, sms, (cudaStream_t)stream);
}

}  // extern "C"
